// Grouped-query attention of few new tokens a sequence (at most 32 rows of (token, head) per kv head).
//
// Bound by HBM where contexts are long (4 x 128k rows, 64 query and 8 kv heads of 128: e4m3 164 us, 6.3 TB/s, bf16
// 295, 7.0), by its warps' chains of instructions where they are ragged and shorter (32 x 8k e4m3 63 us, 4.8 TB/s, bf16
// 100, 6.0).  The pairs of times beside the rules below are those of the step that chose them.  Every visible row of the
// cache is read once for all rows of its kv head, and these together are far below the tensor cores' rate, so the
// products run on warp-level MMAs from registers (tcgen05 would spend 128 rows on at most 32) and the design is
// about the stream of rows:
//  - The visible rows of all (sequence, kv head) units form one list of stages (16 rows, e4m3 32) that is cut into
//    equal pieces, one per CTA, whatever the lengths; a unit cut by a piece's border leaves partial
//    results that a second kernel merges.
//  - A warp takes up to 16 rows of (token, head).  The one or two warps that hold a unit's rows share their stages in a
//    ring of cp.async copies, with one barrier of theirs a stage; these groups stream their own stages and keep their
//    own running maximum, sum and output: no barrier between them until a unit ends.  (All 32 rows in one warp took
//    two CTAs' registers of three, each warp waiting on its own chain of MMAs: at 32 rows a kv head, 48 sequences of
//    up to 4000 rows, 4 kv heads of 128, e4m3 142 us and 102 so, capped bf16 in a window of 1024 41.7 and 38.1; plain
//    bf16 67 and 73.  8 rows a warp, four warps a group: e4m3 111 us, and 16 rows of 64-wide heads 28 for 21 us.)
//  - S = Q K^T has the rows of a kv head as its M (16) and 8 cache rows as its N; its result is, register
//    for register, the A operand of O += P V.  The order of a contraction's terms is free, so a lane
//    reads 16 contiguous bytes of a row and Q's fragments are laid out to match; for P V a lane holds 16
//    contiguous dims of the four rows it needs, and one byte permute a register pairs two rows' codes.
//  - e4m3 caches are never expanded: keys and values enter the MMAs (k32, four times the fp16 rate of these
//    MMAs) as they are, and what meets them is split into two e4m3 terms, x = hi + lo / 2^s, with a sum each.  With at
//    most 8 rows the two terms are the two halves of the MMA's 16 rows, and the second one costs nothing.
//      Queries, brought to at most 448 by a power of two a row, s = 4: a bf16 query's 8 bits are hi's 4 and lo's
//      4, exact down to 2^-15 of the row's largest element, off by 2^-23 of it at most below that.
//      Weights, taken against the stage's own maximum and scaled to at most 256, s = 5: off by 2^-8 of themselves or
//      2^-23 of the stage's largest; the stage's product is added to the running fp32 output with its factor, so a
//      flat tail behind one large weight keeps its precision.
//    A page's V exponent goes onto its product in fp32, apart from the weights' rounding, so a page whose scale is far
//    above the others' takes nothing from them, seen or not.  Two pages of 16 rows in one stage share a product while
//    their exponents lie within NEAR_EXP of one another (the lower one's weights are then off by 2^-19 of the stage's
//    largest, at most); else the stage is gone through once for each of them.
//    The values' bytes are transposed in registers, 4 rows by 4 dims with 8 byte permutes.
//  - bf16 caches: P is rounded to bf16, against a maximum that moves when it is exceeded by more than 2^8.
#include <cooperative_groups.h>

#include "gqa_attention.cuh"
#include "tmap.h"

namespace cg = cooperative_groups;

namespace dsv4 {

static __device__ unsigned int g_flags_gd = 0;

namespace gqa {

namespace dec {

constexpr int NW = 4, THREADS = 32 * NW;
// Sequences whose stages are cut evenly; above, a CTA takes a whole unit: they even out by their number, and every CTA
// would sum up all lengths (1100 sequences of up to 300 e4m3 rows 172 us, 183 as a list; of up to 1500 rows 360 and 387, with
// one kv head of 64 60 and 71; 2000 of up to 4000 rows of that 203 and 215).
constexpr int MAX_SCAN = 1024;
constexpr int MAX_CLUSTER = 8;     // CTAs of a unit (portable cluster size)
constexpr int MIN_ROWS = 128;      // rows of a piece, at least
// rows of a cluster's CTA, at most (16 sequences of up to 2000 e4m3 rows 21.7 us, 23.8 at 512; up to 4000 rows 32, 43 at 2048)
constexpr int CLUSTER_ROWS = 1024;
// Stages that a unit's start and end (lengths, queries, the drained and refilled rings, its merge) weigh in the list: pieces
// of many short units end with those of few long ones (128 sequences of 100 to 1000 e4m3 rows, 8 kv heads: 63 us at 0, 51 at
// 5, 48 at 8 and 12, 49 at 18; 32 x 8k 68.7, 66.4, 65.1 at 12, 66.1 at 18).
constexpr int UNIT_COST = 12;
constexpr float LAZY = 8.f;        // a running maximum moves when it is exceeded by more than 2^8
constexpr int NEAR_EXP = 4;        // V exponents of one product

// Caches: bf16, e4m3, and e4m3 in pages of 16 rows, two of them a stage.  (Pages of 64 rows as if they were two a
// stage: 4 x 128k rows 182 us for 165, 32 x 8k 68.3 for 64.7.)
enum Kind { BF, E4, E4P16 };

struct Args {
  dsv4_gqa_attention_params p;
  float* o_part;    // [2 G][rows][D]
  float2* ml_part;  // [2 G][rows]: maximum of the logits (log2 units), sum
  int4* unit;       // [B * heads]: first and last CTA of the unit, slot in the first, 0 / 1 = merge
  int G, rows;      // CTAs, rows of a partial
  int cs;           // 0: equal pieces of the list; else CTAs (a cluster) of each unit
};

// Shared memory and CTAs per SM: 8 to 16 warps an SM, each with at least 8 KB of copies in flight
// (about 46 KB an SM cover the latency at the full rate), as registers allow (16 rows of e4m3, 128 wide, on three
// CTAs' registers: 75 us where two take 61, at 48 x 4000 rows, 4 kv heads, 16 rows a kv head).
__host__ __device__ constexpr int ctas_per_sm(int D, bool e4m3, int HB) {
  return D == 128 && e4m3 && HB == 2 ? 2 : D == 64 && HB == 1 ? 4 : 3;
}

template <int D, Kind KIND, int HB, int PW, int CTAS>
struct Cfg {
  static constexpr bool E4M3 = KIND != BF;
  static constexpr int ROWB = E4M3 ? D : 2 * D;
  static constexpr int SR = E4M3 ? 32 : 16;    // rows of a stage: an MMA's K
  static constexpr int PG = KIND == E4P16 ? 2 : 1, PB = SR / PG;  // its pages, their rows
  static constexpr int STAGE = 2 * SR * ROWB;  // K then V
  static constexpr int RING = CTAS == 4 ? 12288 : CTAS == 3 ? 16384 : 24576;  // of a warp; a group's are one
  static constexpr int NST = PW * RING / STAGE;
  static constexpr int SMEM = NW * RING;
  static_assert(NST >= 2, "at least one stage ahead");
  static_assert(8 * HB * D * 4 <= RING, "a warp's output fits its ring");
};

struct Shared {
  float m[NW][16], l[NW][16];
  float2 cml[32];     // cluster: this CTA's (maximum, sum) of each row
  int2 meta[NW][32];  // [group][page of the ring]: usable, (k exponent byte | v exponent byte << 8)
};

// c += a b (m16n8k16), bf16.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a b (m16n8k32), e4m3; and c = a b.
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two terms of four values |x| <= 448: x = hi + lo / f, f a power of two.
__device__ __forceinline__ uint2 split_e4m3(float x0, float x1, float x2, float x3, float f) {
  const uint32_t h0 = float2_to_e4m3x2(x0, x1), h1 = float2_to_e4m3x2(x2, x3);
  const float2 f0 = e4m3x2_to_float2((uint16_t)h0), f1 = e4m3x2_to_float2((uint16_t)h1);
  const uint32_t l0 = float2_to_e4m3x2((x0 - f0.x) * f, (x1 - f0.y) * f);
  const uint32_t l1 = float2_to_e4m3x2((x2 - f1.x) * f, (x3 - f1.y) * f);
  return make_uint2(h0 | (h1 << 16), l0 | (l1 << 16));
}
constexpr float QF = 16.f, PF = 32.f;  // 2^s of queries and weights

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Byte offset of 16-byte chunk ch of row r in a stage's K or V half: the chunks of a 128-byte line (one
// row, half of one, or two) are exchanged so that the share-warps of both read patterns (rows 2k, 2k + 1
// with chunks c; rows 2c with the chunks of two lane groups) meet eight different ones.
template <int ROWB>
__device__ __forceinline__ int chunk_at(int r, int ch) {
  if (ROWB == 64) {
    const int line = r >> 1;
    return line * 128 + (((((r & 1) << 2) | ch) ^ (((line & 1) << 2) | (line & 2))) << 4);
  }
  return r * ROWB + ((ch ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
}

struct Unit {
  Seq s;
  int lo, stages;  // first row read (a multiple of SR), stages (0: nothing to do)
  int vlo;         // first row any token sees (the number of rows: none sees any)
};

template <int SR>
__device__ __forceinline__ Unit unit_of(const dsv4_gqa_attention_params& p, int b) {
  Unit u;
  u.s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  u.stages = 0;
  u.lo = u.vlo = 0;
  if (!u.s.ok || u.s.n == 0) return u;
  if (p.kv_start) {
    u.vlo = u.s.kv;
    for (int i = 0; i < u.s.n; ++i) {
      const int2 v = visible_rows(p, b, u.s.t0 + i, u.s.kv - u.s.n + i, u.s.kv);
      if (v.x < v.y) u.vlo = min(u.vlo, v.x);
    }
  } else if (p.window > 0) {
    u.vlo = max(0, u.s.kv - u.s.n - p.window + 1);
  }
  u.lo = u.vlo & ~(SR - 1);
  u.stages = max(1, (u.s.kv - u.lo + SR - 1) / SR);  // (one empty stage where nothing is visible)
  return u;
}

template <int D, Kind KIND, int HB, int PW, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) decode_kernel(Args a) {
  using C = Cfg<D, KIND, HB, PW, CTAS>;
  constexpr bool E4M3 = C::E4M3;
  constexpr int RW = 8 * HB, NG = NW / PW;               // rows of a warp; groups of warps with stages of their own
  constexpr int NT = D / 8, SR = C::SR, PG = C::PG, PB = C::PB;
  constexpr int KS = E4M3 ? D / 32 : D / 16;             // K steps of Q K^T
  constexpr int NQ = E4M3 && HB > 1 ? 2 * KS : KS;       // A fragments of an MMA tile of Q (two terms apart)
  extern __shared__ __align__(1024) uint8_t ring_all[];
  __shared__ Shared sm;
  const dsv4_gqa_attention_params& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int gw = warp / PW, mw = warp % PW;  // group, member
  uint8_t* ring = ring_all + gw * PW * C::RING;
  pdl_wait();
  pdl_launch_dependents();

  // ---------------- this CTA's piece of the list of stages
  int64_t first, last;  // [first, last) in the list
  int b;
  int64_t per;
  int64_t base;  // list position of unit (b, 0)
  if (a.cs == 0) {
    int64_t* pre = reinterpret_cast<int64_t*>(ring_all);  // [B + 1] stages of the sequences before
    int64_t* wsum = pre + MAX_SCAN + 1;
    int64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int bb = b0 + tid;
      int st = 0;
      if (bb < p.B) {
        const Unit u = unit_of<SR>(p, bb);
        st = u.stages ? u.stages + UNIT_COST : 0;
        if (blockIdx.x == 0 && st == 0) {
          if (!u.s.ok) atomicOr(&g_flags_gd, FLAG_PAGE);
          for (int k = 0; k < p.kv_heads; ++k) a.unit[(int64_t)bb * p.kv_heads + k] = make_int4(0, 0, 0, 0);
        }
      }
      int64_t x = st;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) wsum[warp] = x;
      __syncthreads();
      int64_t off = run;
      for (int w = 0; w < warp; ++w) off += wsum[w];
      if (bb < p.B) pre[bb] = off + x - st;
      for (int w = 0; w < NW; ++w) run += wsum[w];
      __syncthreads();
    }
    const int64_t total = run * p.kv_heads;
    per = (total + a.G - 1) / a.G;
    if (per < MIN_ROWS / SR) per = MIN_ROWS / SR;
    first = (int64_t)blockIdx.x * per;
    last = min(total, first + per);
    if (first >= last) return;
    int lo = 0, hi = p.B;  // the last b whose list position is <= first (empty sequences share one: the last)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] * p.kv_heads <= first) lo = mid;
      else hi = mid;
    }
    b = lo;
    base = pre[b] * p.kv_heads;
    __syncthreads();
  } else {
    // a unit's stages in even pieces over the CTAs of a cluster
    const int unit = blockIdx.x / a.cs, rank = blockIdx.x % a.cs;
    b = unit / p.kv_heads;
    const Unit u = unit_of<SR>(p, b);
    if (u.stages == 0) {
      if (tid == 0 && rank == 0 && !u.s.ok) atomicOr(&g_flags_gd, FLAG_PAGE);
      return;
    }
    base = 0;
    per = (u.stages + a.cs - 1) / a.cs;
    first = (int64_t)(unit % p.kv_heads) * u.stages;
    last = first + min((int64_t)u.stages, (rank + 1) * per);
    first += min((int64_t)u.stages, rank * per);
    if (tid < 32) sm.cml[tid] = make_float2(-INFINITY, 0.f);
    __syncthreads();
  }

  const int group = p.q_heads / p.kv_heads;
  const bool plain = p.softcap == 0.f && p.slopes == nullptr;
  const int cost = a.cs ? 0 : UNIT_COST;
  const float rcap2 = p.softcap > 0.f ? 2.f * LOG2E / p.softcap : 0.f;

  // ---------------- the units that the piece meets
  for (int64_t at = first; at < last; ++b) {
    const Unit u = unit_of<SR>(p, b);
    if (u.stages == 0) continue;
    const int weight = u.stages + cost;
    for (int h = (int)((at - base) / weight); h < p.kv_heads && at < last; ++h) {
      const int64_t u0 = base + (int64_t)h * weight;  // the unit's list positions [u0, u0 + weight), its cost's first
      const int64_t end = min(last, u0 + weight);
      const int s0 = (int)max(at - u0 - cost, (int64_t)0), s1 = (int)(end - u0) - cost;
      if (s1 <= s0) {  // none of its stages is here
        at = end;
        continue;
      }
      const bool whole = a.cs == 1 || (a.cs == 0 && s0 == 0 && s1 == u.stages);
      const int rows = u.s.n * group, row0 = RW * mw;  // the unit's, this warp's first
      const int pos0 = u.s.kv - u.s.n;

      // rows g + 8 k of this lane
      int rlo[HB], rhi[HB];
      float rmul[HB], slope[HB];
      int rpos[HB];
      float m[HB], l[HB];
      int all_lo = 0, all_hi = 0x7FFFFFFF;  // rows that every token sees
      // Q's A fragments; e4m3: [K step][hi, lo], or both terms in one for 8 rows.
      uint32_t q[NQ][4];
      auto keep_q = [&](int x, int k, uint32_t lo, uint32_t hi) {  // fragment x, row half k
        q[x][k] = lo;
        q[x][2 + k] = hi;
      };
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        const int r = row0 + g + 8 * k, i = r / group;
        const bool live = r < rows;
        const int pos = pos0 + i, t = u.s.t0 + i;
        rlo[k] = 0;
        rhi[k] = 0;
        slope[k] = 0.f;
        rpos[k] = pos;
        rmul[k] = 0.f;
        m[k] = -INFINITY;
        l[k] = 0.f;
        const int head = h * group + r % group;
        if (live) {
          const int2 v = visible_rows(p, b, t, pos, u.s.kv);
          rlo[k] = v.x;
          rhi[k] = v.y;
          if (p.slopes) slope[k] = p.slopes[head] * LOG2E;
          all_lo = max(all_lo, v.x);
          all_hi = min(all_hi, v.y);
        }
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q) +
                             2 * ((int64_t)t * p.q_token_stride + (int64_t)head * p.q_head_stride);
        float mul = p.softmax_scale;
        if (E4M3) {
          // the 8 dims of K step s (of 32) that this lane's K registers hold, split in two terms
          uint4 w[KS];
          float big = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            w[s] = live ? *reinterpret_cast<const uint4*>(src + 2 * (64 * (s / 2) + 16 * c + 8 * (s % 2))) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t ww[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              big = fmaxf(big, fmaxf(fabsf(__uint_as_float(ww[y] << 16)), fabsf(__uint_as_float(ww[y] & 0xFFFF0000u))));
          }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int e = ue8m0_exponent(big);
          const float f = exp2_neg_int(e);
          mul *= exp2_neg_int(-e);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const uint32_t ww[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
            float v[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              v[2 * y] = __uint_as_float(ww[y] << 16) * f;
              v[2 * y + 1] = __uint_as_float(ww[y] & 0xFFFF0000u) * f;
            }
            const uint2 u0 = split_e4m3(v[0], v[1], v[2], v[3], QF), u1 = split_e4m3(v[4], v[5], v[6], v[7], QF);
            if (HB == 1) {  // (rows 0-7: hi, rows 8-15: lo)
              keep_q(s, 0, u0.x, u1.x);
              keep_q(s, 1, u0.y, u1.y);
            } else {
              keep_q(2 * s, k, u0.x, u1.x);
              keep_q(2 * s + 1, k, u0.y, u1.y);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < KS; ++s) {  // the 4 dims of K step s (of 16)
            const uint2 w = live ? *reinterpret_cast<const uint2*>(src + 2 * (32 * (s / 2) + 8 * c + 4 * (s % 2))) : make_uint2(0u, 0u);
            keep_q(s, k, w.x, w.y);
            if (HB == 1) keep_q(s, 1, 0u, 0u);
          }
        }
        rmul[k] = plain ? mul * LOG2E : mul;
      }
      all_lo = __reduce_max_sync(0xffffffffu, all_lo);
      all_hi = __reduce_min_sync(0xffffffffu, all_hi);

      // the running output: row half k, column tile j, columns 2c and 2c + 1.  bf16: the MMAs' accumulators
      float o[E4M3 ? HB : 1][NT][E4M3 ? 2 : 4];
#pragma unroll
      for (auto& x : o)
#pragma unroll
        for (auto& y : x)
#pragma unroll
          for (float& v : y) v = 0.f;
      auto out = [&](int k, int j, int y) -> float& { return E4M3 ? o[k][j][y] : o[0][j][2 * k + y]; };

      // this group's stages: s0 + gw, s0 + gw + NG, ...
      const int count = s1 - s0 > gw ? (s1 - s0 - gw + NG - 1) / NG : 0;
      int pid = -1, pexp = 0;
      constexpr int CPR = C::ROWB / 16, RPI = 32 * PW / CPR;  // lanes of a row, rows the group copies at once
      constexpr int NU = SR / RPI;                            // 16-byte pieces of K (and V) that a thread copies
      constexpr int64_t ES = E4M3 ? 1 : 2;
      static_assert(NU * RPI == SR, "whole rounds");
      const int gl = mw * 32 + lane, r_in = gl / CPR;
      const uint8_t* k_base = reinterpret_cast<const uint8_t*>(p.k_cache) + ES * ((int64_t)h * p.k_cache_head_stride) + 16 * (gl % CPR);
      const uint8_t* v_base = reinterpret_cast<const uint8_t*>(p.v_cache) + ES * ((int64_t)h * p.v_cache_head_stride) + 16 * (gl % CPR);
      const int64_t k_step = ES * RPI * p.k_row_stride, v_step = ES * RPI * p.v_row_stride;
      int doff[NU];
#pragma unroll
      for (int i = 0; i < NU; ++i) doff[i] = chunk_at<C::ROWB>(i * RPI + r_in, gl % CPR);
      auto fill = [&](int k) {
        if (k < count) {
          if ((k * PG & 31) == 0) {  // the next 32 pages and their exponents, one a lane
            const int ks = k + lane / PG, j = u.lo + (s0 + gw + ks * NG) * SR + lane % PG * PB;
            pid = -1;
            pexp = 0;
            if (ks < count && j + PB > u.vlo && j < u.s.kv) {  // (pages that no token sees are not looked at)
              const int lp = j / p.page_size;
              pid = lp < p.max_pages_per_seq ? p.block_table[(int64_t)b * p.max_pages_per_seq + lp] : -1;
              if (pid < 0 || pid >= p.num_pages) {
                atomicOr(&g_flags_gd, FLAG_PAGE);
                pid = -1;
              } else if (E4M3) {
                const int64_t e = (int64_t)pid * p.kv_heads + h;
                pexp = (int)p.k_exp[e] | ((int)p.v_exp[e] << 8);
              }
            }
          }
          const int slot = k % C::NST, js = u.lo + (s0 + gw + k * NG) * SR;
          uint8_t* dst = ring + slot * C::STAGE;
          constexpr int PER = RPI < PB ? PB / RPI : 1;  // pieces that a thread copies of a page
          static_assert(NU % PER == 0 && C::NST * PG <= 32, "whole pages; the ring's lie in sm.meta");
#pragma unroll
          for (int y = 0; y < PG; ++y) {
            const int page = __shfl_sync(0xffffffffu, pid, (k * PG + y) & 31);
            const int ex = __shfl_sync(0xffffffffu, pexp, (k * PG + y) & 31);
            if (mw == 0 && lane == 0) sm.meta[gw][slot * PG + y] = make_int2(page >= 0, ex);
          }
#pragma unroll
          for (int nb = 0; nb < NU; nb += PER) {
            const int rb = nb * RPI + r_in;  // the first of PER rows in one page
            const int page = __shfl_sync(0xffffffffu, pid, (k * PG + rb / PB) & 31);
            const int j0 = js + rb;
            const int row = j0 & (p.page_size - 1);
            const uint8_t* kr = k_base + ES * ((int64_t)max(page, 0) * p.k_page_stride + (int64_t)row * p.k_row_stride);
            const uint8_t* vr = v_base + ES * ((int64_t)max(page, 0) * p.v_page_stride + (int64_t)row * p.v_row_stride);
            const int jb = j0 & ~(PB - 1);
            if (page >= 0 && jb >= u.vlo && jb + PB <= u.s.kv) {
#pragma unroll
              for (int i = 0; i < PER; ++i) {
                tc::cp_async16(dst + doff[nb + i], kr + i * k_step, 16u);
                tc::cp_async16(dst + SR * C::ROWB + doff[nb + i], vr + i * v_step, 16u);
              }
            } else {
              // rows that no token sees read nothing and become zeros, whatever the cache holds there
#pragma unroll
              for (int i = 0; i < PER; ++i) {
                const int j = j0 + i * RPI;
                const bool in = page >= 0 && j >= u.vlo && j < u.s.kv;
                tc::cp_async16(dst + doff[nb + i], in ? kr + i * k_step : reinterpret_cast<const uint8_t*>(p.k_cache), in ? 16u : 0u);
                tc::cp_async16(dst + SR * C::ROWB + doff[nb + i], in ? vr + i * v_step : reinterpret_cast<const uint8_t*>(p.v_cache),
                               in ? 16u : 0u);
              }
            }
          }
        }
        tc::cp_async_commit();
      };
      auto group_sync = [&]() {
        if (PW == 1) __syncwarp();
        else tc::named_bar_sync(1 + gw, 32 * PW);
      };
#pragma unroll 1
      for (int k = 0; k < C::NST - 1; ++k) fill(k);

      // only -1: the stage's rows together; 0, then 1: those of one page (V exponents too far apart for one product)
      int only = -1;
#pragma unroll 1
      for (int k = 0; k < count;) {
        if (PG == 1 || only != 0) {
          tc::cp_async_wait<C::NST - 2>();
          group_sync();  // the stage is there for all, and the one before is read
          fill(k + C::NST - 1);
        }
        if (row0 >= rows) {  // a warp with no rows only copies
          ++k;
          continue;
        }
        const int slot = k % C::NST, j0 = u.lo + (s0 + gw + k * NG) * SR;
        const uint8_t* kt = ring + slot * C::STAGE;
        const uint8_t* vt = kt + SR * C::ROWB;

        if (PG > 1) {
          const int2 m0 = sm.meta[gw][slot * PG], m1 = sm.meta[gw][slot * PG + PG - 1];
          only = only == 0 ? 1 : m0.x && m1.x && abs((m0.y >> 8) - (m1.y >> 8)) > NEAR_EXP ? 0 : -1;
        }
        // ---- S = Q K^T: z[row half][tile of 8 rows][row 2c, 2c + 1 of it]
        float z[HB][SR / 8][2];
#pragma unroll
        for (int nt = 0; nt < SR / 8; ++nt) {
          constexpr int KCH = C::ROWB / 64;  // 16-byte chunks a lane holds of a row
          float s[4], s_lo[4];
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            const uint4 w = *reinterpret_cast<const uint4*>(kt + chunk_at<C::ROWB>(8 * nt + g, c + 4 * x));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int ks = 2 * x + y;
              if (E4M3) {
                const int f = HB == 1 ? ks : 2 * ks;
                if (ks == 0) mma8_first(s, q[f], ww[2 * y], ww[2 * y + 1]);
                else mma8(s, q[f], ww[2 * y], ww[2 * y + 1]);
                if (HB > 1) {
                  if (ks == 0) mma8_first(s_lo, q[f + 1], ww[2 * y], ww[2 * y + 1]);
                  else mma8(s_lo, q[f + 1], ww[2 * y], ww[2 * y + 1]);
                }
              } else {
                if (ks == 0) s[0] = s[1] = s[2] = s[3] = 0.f;
                mma16(s, q[ks], ww[2 * y], ww[2 * y + 1]);
              }
            }
          }
#pragma unroll
          for (int k2 = 0; k2 < HB; ++k2)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int e = 2 * k2 + y;
              z[k2][nt][y] = !E4M3 ? s[e] : HB == 1 ? fmaf(s[2 + y], 1.f / QF, s[y]) : fmaf(s_lo[e], 1.f / QF, s[e]);
            }
        }

        // ---- logits in log2 units, masks, the stage's maximum of each row (this lane's part)
        float top[HB];
        int vbyte[PG];
        bool inside = j0 >= all_lo && j0 + SR <= all_hi;
        float kmul[PG];
        bool page_ok[PG];
#pragma unroll
        for (int y = 0; y < PG; ++y) {
          const int2 meta = sm.meta[gw][slot * PG + y];
          page_ok[y] = meta.x != 0 && (PG == 1 || only < 0 || only == y);
          inside = inside && page_ok[y];
          kmul[y] = E4M3 ? ue8m0_scale((uint8_t)(meta.y & 255)) : 1.f;
          vbyte[y] = meta.y >> 8;
        }
#pragma unroll
        for (int k2 = 0; k2 < HB; ++k2) {
          top[k2] = -INFINITY;
          const float far = (float)(rpos[k2] - j0 - 2 * c);  // (near distances stay exact however long the cache)
#pragma unroll
          for (int nt = 0; nt < SR / 8; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float& v = z[k2][nt][y];
              v = E4M3 ? v * kmul[nt * 8 / PB] * rmul[k2] : v * rmul[k2];
              const int j = j0 + 8 * nt + 2 * c + y;
              if (!plain) {
                if (p.softcap > 0.f) v = cap_logit(v, p.softcap, rcap2);
                v = v * LOG2E - slope[k2] * fabsf(far - (float)(8 * nt + y));
              }
              if (!inside && (!page_ok[nt * 8 / PB] || j < rlo[k2] || j >= rhi[k2])) v = -INFINITY;
              top[k2] = fmaxf(top[k2], v);
            }
        }

        if (E4M3) {
          // ---- weights against the stage's maximum, in two e4m3 terms; its V exponent
          int vtop = vbyte[0];
          float vf[PG];  // a page's weights in its product
          if (PG > 1) {
            vtop = max(page_ok[0] ? vbyte[0] : 0, page_ok[PG - 1] ? vbyte[PG - 1] : 0);
#pragma unroll
            for (int y = 0; y < PG; ++y) vf[y] = page_ok[y] ? exp2_neg_int(vtop - vbyte[y]) : 0.f;
          }
          const float vscale = ue8m0_scale((uint8_t)vtop);
          uint32_t hi[HB][2], lo[HB][2];
          float fs[HB];
          bool move = false;
          float fo[HB];
#pragma unroll
          for (int k2 = 0; k2 < HB; ++k2) {
            float t = top[k2];
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
            const float ref = (t == -INFINITY ? 0.f : t) - 8.f;  // (weights of at most 256, and their sum so)
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < SR / 8; ++nt)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float& v = z[k2][nt][y];
                v = tc::ex2_approx(v - ref);
                sum += v;
                if (PG > 1) v *= vf[nt * 8 / PB];
              }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint2 w = split_e4m3(z[k2][2 * x][0], z[k2][2 * x][1], z[k2][2 * x + 1][0], z[k2][2 * x + 1][1], PF);
              hi[k2][x] = w.x;
              lo[k2][x] = w.y;
            }
            const float mn = fmaxf(m[k2], t), mr = mn == -INFINITY ? 0.f : mn;
            fo[k2] = tc::ex2_approx(m[k2] - mr);
            const float ft = tc::ex2_approx(t - mr) * 0x1p-8f;
            l[k2] = fmaf(l[k2], fo[k2], sum * ft);
            fs[k2] = ft * vscale;
            move |= mn > m[k2];
            m[k2] = mn;
          }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int k2 = 0; k2 < HB; ++k2)
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                out(k2, j, 0) *= fo[k2];
                out(k2, j, 1) *= fo[k2];
              }
          }
          // ---- O += P V: 4 dims (a word of the lane's) at a time
          constexpr int WD = D / 32;
          uint32_t v[8][WD];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = 2 * c + (y & 1) + 8 * (y >> 1);
            if (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(vt + chunk_at<C::ROWB>(r, (g >> 1) | ((g & 1) << 2)));
              v[y][0] = w.x;
              v[y][1] = w.y;
              v[y][WD - 2] = w.z;
              v[y][WD - 1] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(vt + chunk_at<C::ROWB>(r, g >> 1) + 8 * (g & 1));
              v[y][0] = w.x;
              v[y][1] = w.y;
            }
          }
#pragma unroll
          for (int wd = 0; wd < WD; ++wd) {
            uint32_t bt[2][4];  // [rows 0-15, 16-31 of the stage][dim]: four rows' codes of one dim
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t t0 = __byte_perm(v[4 * x][wd], v[4 * x + 1][wd], 0x5140u);
              const uint32_t t1 = __byte_perm(v[4 * x][wd], v[4 * x + 1][wd], 0x7362u);
              const uint32_t u0 = __byte_perm(v[4 * x + 2][wd], v[4 * x + 3][wd], 0x5140u);
              const uint32_t u1 = __byte_perm(v[4 * x + 2][wd], v[4 * x + 3][wd], 0x7362u);
              bt[x][0] = __byte_perm(t0, u0, 0x5410u);
              bt[x][1] = __byte_perm(t0, u0, 0x7632u);
              bt[x][2] = __byte_perm(t1, u1, 0x5410u);
              bt[x][3] = __byte_perm(t1, u1, 0x7632u);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const int j = 4 * wd + d;
              if (HB == 1) {
                const uint32_t f[4] = {hi[0][0], lo[0][0], hi[0][1], lo[0][1]};
                float x[4];
                mma8_first(x, f, bt[0][d], bt[1][d]);
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  out(0, j, y) = fmaf(fmaf(x[2 + y], 1.f / PF, x[y]), fs[0], out(0, j, y));
              } else {
                constexpr int k1 = HB - 1;
                const uint32_t f[4] = {hi[0][0], hi[k1][0], hi[0][1], hi[k1][1]};
                const uint32_t f2[4] = {lo[0][0], lo[k1][0], lo[0][1], lo[k1][1]};
                float x[4], x2[4];
                mma8_first(x, f, bt[0][d], bt[1][d]);
                mma8_first(x2, f2, bt[0][d], bt[1][d]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  out(0, j, y) = fmaf(fmaf(x2[y], 1.f / PF, x[y]), fs[0], out(0, j, y));
                  out(k1, j, y) = fmaf(fmaf(x2[2 + y], 1.f / PF, x[2 + y]), fs[k1], out(k1, j, y));
                }
              }
            }
          }
        } else {
          // ---- running maxima: moved (by the whole quad) only when some logit exceeds one by more than LAZY
          bool move = false;
#pragma unroll
          for (int k2 = 0; k2 < HB; ++k2) move |= top[k2] > m[k2] + LAZY;
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int k2 = 0; k2 < HB; ++k2) {
              float t = top[k2];
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
              const float mn = fmaxf(m[k2], t);
              const float f = m[k2] == -INFINITY ? 0.f : tc::ex2_approx(m[k2] - mn);
              l[k2] *= f;
              m[k2] = mn;
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                out(k2, j, 0) *= f;
                out(k2, j, 1) *= f;
              }
            }
          }
          uint32_t pa[4];
          if (HB == 1) pa[1] = pa[3] = 0u;
#pragma unroll
          for (int k2 = 0; k2 < HB; ++k2) {
            const float mm = m[k2] == -INFINITY ? 0.f : m[k2];
            float w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = tc::ex2_approx(z[k2][y >> 1][y & 1] - mm);
            l[k2] += (w[0] + w[1]) + (w[2] + w[3]);
            pa[k2] = float2_to_bf16x2_bits(w[0], w[1]);
            pa[2 + k2] = float2_to_bf16x2_bits(w[2], w[3]);
          }
          // ---- O += P V; the matrices of an x4 load: rows 0-7 and 8-15 of dims 16 jj .. + 7, then of the next 8
          const int r = (lane & 7) + (lane & 8);
#pragma unroll
          for (int jj = 0; jj < NT / 2; ++jj) {
            uint32_t w[4];
            ldmatrix_x4_trans(w, tc::smem_addr(vt + chunk_at<C::ROWB>(r, 2 * jj + (lane >> 4))));
            if constexpr (!E4M3) {
              mma16(o[0][2 * jj], pa, w[0], w[1]);
              mma16(o[0][2 * jj + 1], pa, w[2], w[3]);
            }
          }
        }
        if (PG == 1 || only != 0) ++k;
      }
      tc::cp_async_wait<0>();

      // ---------------- the groups' results of the unit
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        if (c == 0) {
          sm.m[warp][g + 8 * k] = m[k];
          sm.l[warp][g + 8 * k] = l[k];
        }
      }
      __syncthreads();
      float* part = reinterpret_cast<float*>(ring_all + warp * C::RING);  // [RW][D]: the rings are drained
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        const int r = g + 8 * k;
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < NG; ++w) mn = fmaxf(mn, sm.m[w * PW + mw][r]);
        const float f = m[k] == -INFINITY ? 0.f : tc::ex2_approx(m[k] - mn);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          // column n of tile j is dim 16 f(n) + j, f(n) the chunk of lane group n (e4m3, D = 128), 8 n + j (D = 64)
          // or 8 j + n (bf16); this lane has columns 2 c and 2 c + 1
          const int d0 = !E4M3 ? 8 * j + 2 * c : D == 128 ? 16 * c + j : 16 * c + j;
          const int d1 = !E4M3 ? d0 + 1 : D == 128 ? d0 + 64 : d0 + 8;
          part[r * D + d0] = out(k, j, 0) * f;
          part[r * D + d1] = out(k, j, 1) * f;
        }
      }
      __syncthreads();
      const int slot = 2 * blockIdx.x + (at == first ? 0 : 1);
      for (int x = tid; x < rows * (D / 4); x += THREADS) {
        const int r = x / (D / 4), d4 = x % (D / 4);
        const int rm = r / RW, rl = r % RW;  // the row's warp in a group, its place there
        float mn = -INFINITY, ls = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          mn = fmaxf(mn, sm.m[w * PW + rm][rl]);
          const float4 v = reinterpret_cast<const float4*>(ring_all + (w * PW + rm) * C::RING)[rl * (D / 4) + d4];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
#pragma unroll
        for (int w = 0; w < NG; ++w)
          if (sm.m[w * PW + rm][rl] > -INFINITY) ls += sm.l[w * PW + rm][rl] * tc::ex2_approx(sm.m[w * PW + rm][rl] - mn);
        if (whole) {
          const int head = h * group + r % group;
          const int64_t row = (int64_t)(u.s.t0 + r / group) * p.q_heads + head;
          const float f = finish_scale(p, row, head, mn, ls, d4 == 0);
          store4<D>(p, row, d4, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
        } else if (a.cs) {
          reinterpret_cast<float4*>(ring_all + rm * C::RING)[rl * (D / 4) + d4] = acc;  // (over group 0's, which this thread has read)
          if (d4 == 0) sm.cml[r] = make_float2(mn, ls);
        } else {
          reinterpret_cast<float4*>(a.o_part)[((int64_t)slot * a.rows + r) * (D / 4) + d4] = acc;
          if (d4 == 0) a.ml_part[(int64_t)slot * a.rows + r] = make_float2(mn, ls);
        }
      }
      if (tid == 0 && s0 == 0 && a.cs == 0)
        a.unit[(int64_t)b * p.kv_heads + h] =
            whole ? make_int4(0, 0, 0, 0)
                  : make_int4((int)blockIdx.x, (int)((u0 + weight - 1) / per), at == first ? 0 : 1, 1);
      __syncthreads();
      at = end;
    }
    base += (int64_t)p.kv_heads * weight;
  }

  if (a.cs > 1) {
    // ---------------- the cluster's pieces of the unit, joined through distributed shared memory: every CTA finishes
    // its share of the output
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int unit = blockIdx.x / a.cs, rank = blockIdx.x % a.cs;
    const Unit u = unit_of<SR>(p, unit / p.kv_heads);
    const int h = unit % p.kv_heads, rows = u.s.n * group;
    for (int x = rank * THREADS + tid; x < rows * (D / 4); x += a.cs * THREADS) {
      const int r = x / (D / 4), d4 = x % (D / 4);
      float2 ml[MAX_CLUSTER];
      float4 v[MAX_CLUSTER];
      float mn = -INFINITY, ls = 0.f;
#pragma unroll
      for (int i = 0; i < MAX_CLUSTER; ++i) {  // (all at once: one latency)
        ml[i] = make_float2(-INFINITY, 0.f);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < a.cs) {
          ml[i] = cl.map_shared_rank(sm.cml, i)[r];
          v[i] = cl.map_shared_rank(reinterpret_cast<float4*>(ring_all + r / RW * C::RING), i)[r % RW * (D / 4) + d4];
        }
      }
#pragma unroll
      for (int i = 0; i < MAX_CLUSTER; ++i) mn = fmaxf(mn, ml[i].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < MAX_CLUSTER; ++i) {
        if (ml[i].x == -INFINITY) continue;  // (a piece without visible rows: its sums may not have been written)
        const float f = tc::ex2_approx(ml[i].x - mn);
        ls = fmaf(ml[i].y, f, ls);
        acc.x = fmaf(v[i].x, f, acc.x);
        acc.y = fmaf(v[i].y, f, acc.y);
        acc.z = fmaf(v[i].z, f, acc.z);
        acc.w = fmaf(v[i].w, f, acc.w);
      }
      const int head = h * group + r % group;
      const int64_t row = (int64_t)(u.s.t0 + r / group) * p.q_heads + head;
      const float f = finish_scale(p, row, head, mn, ls, d4 == 0);
      store4<D>(p, row, d4, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
    }
    cl.sync();  // no CTA leaves while its shared memory is read
  }
}

// Joins the partial results of the units that a piece's border cuts.  Q warps a row, each with every Qth eight of the
// partials, all eight in flight: 4 where a unit has more than 8 partials on average (one warp a row: one token over
// 16,000 rows 31 us for 22, 4 x 128k rows 180 for 174), else 1 (four: 32 x 8k rows 75 us for 69,
// most of the warps idle).
template <int D, int Q>
__global__ void __launch_bounds__(Q * THREADS) merge_kernel(Args a) {
  __shared__ float4 part[NW][Q][D / 4];
  __shared__ float sums[NW][Q];
  pdl_wait();
  pdl_launch_dependents();
  const dsv4_gqa_attention_params& p = a.p;
  const int4 info = a.unit[blockIdx.x];
  if (info.w == 0) return;
  const int b = blockIdx.x / p.kv_heads, h = blockIdx.x % p.kv_heads, lane = threadIdx.x & 31;
  const int wr = (threadIdx.x >> 5) / Q, share = (threadIdx.x >> 5) % Q, r = blockIdx.y * NW + wr;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  const int group = p.q_heads / p.kv_heads, rows = s.n * group, n = info.y - info.x + 1;
  auto slot = [&](int i) { return (int64_t)(2 * (info.x + i) + (i == 0 ? info.z : 0)) * a.rows + r; };
  float mn = -INFINITY;
  if (r < rows) {
    for (int i = lane; i < n; i += 32) mn = fmaxf(mn, a.ml_part[slot(i)].x);
    mn = warp_max(mn);
    float ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    for (int i0 = U * share; i0 < n; i0 += Q * U) {
      float4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + k < n && lane < D / 4) v[k] = reinterpret_cast<const float4*>(a.o_part)[slot(i0 + k) * (D / 4) + lane];
      }
      float2 x = make_float2(-INFINITY, 0.f);  // lane k's: partial k's
      if (lane < U && i0 + lane < n) x = a.ml_part[slot(i0 + lane)];
      const float f = x.x > -INFINITY ? tc::ex2_approx(x.x - mn) : 0.f;  // (else its sums are zeros)
      ls = fmaf(x.y, f, ls);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k);
        acc.x = fmaf(v[k].x, fk, acc.x);
        acc.y = fmaf(v[k].y, fk, acc.y);
        acc.z = fmaf(v[k].z, fk, acc.z);
        acc.w = fmaf(v[k].w, fk, acc.w);
      }
    }
    ls = warp_sum(ls);
    if (lane < D / 4) part[wr][share][lane] = acc;
    if (lane == 0) sums[wr][share] = ls;
  }
  __syncthreads();
  if (r >= rows || share != 0 || lane >= D / 4) return;
  float ls = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int y = 0; y < Q; ++y) {
    const float4 v = part[wr][y][lane];
    ls += sums[wr][y];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const int head = h * group + r % group;
  const int64_t row = (int64_t)(s.t0 + r / group) * p.q_heads + head;
  const float f = finish_scale(p, row, head, mn, ls, lane == 0);
  store4<D>(p, row, lane, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
}

struct Plan {
  int hb, pw, rows, G, cs;
  size_t ml_off, unit_off, total;
};

// Row halves of 8 that hold the rows of a kv head, and the CTAs: what the device holds at once, or fewer
// where even the largest batch within the call's bounds has fewer pieces of MIN_ROWS.
static Plan plan(const dsv4_gqa_attention_params& p) {
  Plan L;
  const int max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  L.rows = max_n * (p.q_heads / p.kv_heads);
  L.hb = L.rows <= 8 ? 1 : 2;
  L.pw = L.rows <= 16 ? 1 : 2;
  L.rows = 8 * L.hb * L.pw;
  const int ctas = ctas_per_sm(p.head_dim, p.cache_dtype == DSV4_E4M3_PAGE, L.hb);
  const int64_t pieces = ((int64_t)p.B * p.kv_heads * (p.max_kv_len + (2 + UNIT_COST) * 32) + MIN_ROWS - 1) / MIN_ROWS;
  L.G = num_sms() * ctas;
  if (pieces < L.G) L.G = (int)pieces;
  // A cluster a unit where the batch is small enough for all units' clusters to be resident and a warp to have
  // few stages: its join costs less than a second kernel (one token over 777 rows 8.8 us, 10.1 as pieces; 48 x 4
  // tokens in a window of 1024 38 and 42; 200 sequences of up to 1500 rows, one kv head, 21.2 and 22.2).  Else, evenly cut pieces; beyond MAX_SCAN, a CTA a unit.
  const int64_t units = (int64_t)p.B * p.kv_heads;
  int64_t seen = p.max_kv_len;
  if (p.window > 0 && (int64_t)p.window + max_n < seen) seen = (int64_t)p.window + max_n;
  L.cs = p.B > MAX_SCAN ? 1 : 0;
  for (int cs = MAX_CLUSTER; cs >= 2 && L.cs == 0; cs /= 2)
    if (units * cs <= (int64_t)num_sms() * ctas && seen <= (int64_t)CLUSTER_ROWS * cs) L.cs = cs;
  const int64_t slots = L.cs == 0 ? 2LL * L.G : 0;
  L.ml_off = align_up((size_t)slots * L.rows * p.head_dim * 4, 256);
  L.unit_off = align_up(L.ml_off + (size_t)slots * L.rows * 8, 256);
  L.total = align_up(L.unit_off + (size_t)units * 16, 256);
  return L;
}

template <int D, Kind KIND, int HB, int PW, int CTAS>
static cudaError_t launch(const Args& a, cudaStream_t s) {
  using C = Cfg<D, KIND, HB, PW, CTAS>;
  const void* fn = reinterpret_cast<const void*>(decode_kernel<D, KIND, HB, PW, CTAS>);
  cudaError_t e = ensure_max_dynamic_smem(fn, C::SMEM);
  if (e != cudaSuccess) return e;
  const dsv4_gqa_attention_params& p = a.p;
  const int64_t units = (int64_t)p.B * p.kv_heads;
  if (units > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.cs ? (unsigned)(units * a.cs) : a.G);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cs ? a.cs : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = count_launch(cudaLaunchKernelEx(&cfg, decode_kernel<D, KIND, HB, PW, CTAS>, a));
  if (e != cudaSuccess || a.cs) return e;
  const dim3 grid((unsigned)units, a.rows / NW);
  if (a.G > 8 * units) return launch_pdl(merge_kernel<D, 4>, grid, dim3(4 * THREADS), 0, s, true, a);
  return launch_pdl(merge_kernel<D, 1>, grid, dim3(THREADS), 0, s, true, a);
}

// Where at most two CTAs an SM have work, they are built for two: deeper rings, more registers (8 kv heads, 16
// sequences of up to 2000 rows: e4m3 26.5 us for 21.4, bf16 26.5 for 23.2; one token over 6000 bf16 rows 17.2 for 13.4).
template <int D, Kind KIND, int HB, int PW>
static cudaError_t launch_ctas(const Args& a, cudaStream_t s) {
  const int64_t ctas = a.cs ? (int64_t)a.p.B * a.p.kv_heads * a.cs : a.G;
  constexpr int most = ctas_per_sm(D, KIND != BF, HB);
  if (most > 2 && ctas <= 2LL * num_sms()) return launch<D, KIND, HB, PW, 2>(a, s);
  return launch<D, KIND, HB, PW, most>(a, s);
}

template <int D, Kind KIND>
static cudaError_t launch_rows(const Args& a, const Plan& L, cudaStream_t s) {
  if (L.hb == 1) return launch_ctas<D, KIND, 1, 1>(a, s);
  return L.pw == 2 ? launch_ctas<D, KIND, 2, 2>(a, s) : launch_ctas<D, KIND, 2, 1>(a, s);
}

template <int D>
static cudaError_t launch_kind(const Args& a, Kind kind, const Plan& L, cudaStream_t s) {
  if (kind == BF) return launch_rows<D, BF>(a, L, s);
  return kind == E4 ? launch_rows<D, E4>(a, L, s) : launch_rows<D, E4P16>(a, L, s);
}

}  // namespace dec

size_t decode_workspace(const dsv4_gqa_attention_params& p) { return dec::plan(p).total; }

cudaError_t launch_decode(const dsv4_gqa_attention_params& p, cudaStream_t s) {
  const dec::Plan L = dec::plan(p);
  dec::Args a;
  a.p = p;
  uint8_t* ws = reinterpret_cast<uint8_t*>(p.workspace);
  a.o_part = reinterpret_cast<float*>(ws);
  a.ml_part = reinterpret_cast<float2*>(ws + L.ml_off);
  a.unit = reinterpret_cast<int4*>(ws + L.unit_off);
  a.G = L.G;
  a.rows = L.rows;
  a.cs = L.cs;
  const dec::Kind kind = p.cache_dtype != DSV4_E4M3_PAGE ? dec::BF : p.page_size == 16 ? dec::E4P16 : dec::E4;
  return p.head_dim == 128 ? dec::launch_kind<128>(a, kind, L, s) : dec::launch_kind<64>(a, kind, L, s);
}

}  // namespace gqa

cudaError_t read_flags_gqa_decode(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_gd, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_gd, &z, sizeof(z));
}

}  // namespace dsv4
