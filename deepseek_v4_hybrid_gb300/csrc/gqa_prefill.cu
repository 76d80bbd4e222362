// Grouped-query attention of many new tokens a sequence: tcgen05 products with TMEM accumulators.
//
// The rows (token, head of the group) of one kv head, token by token, are cut into units of 256: two MMA
// tiles of 128 rows that share every key and value tile of 128 cache rows.
//   S_i = Q_i K^T          M = 128 rows, N = 128 cache rows, K = head_dim     (shared memory x shared memory)
//   O_i += P_i V           M = 128 rows, N = head_dim, K = 128 cache rows     (tensor memory x shared memory)
// TMEM: S_0, S_1 (128 columns each; P_i as bf16 over the first half of S_i), O_0, O_1.
//   Warps 0-3 and 4-7 (a warpgroup a tile): a thread owns a row: reads S from TMEM, masks, caps, takes the online
//   softmax in log2 units (O is rescaled only when a row's maximum grows by more than 2^8) and writes P back.
//   Warps 8-11 write the output of a finished unit while the softmax is at the next one.
//   Warp 12 loads key and value tiles by TMA (one box a page) into a ring of four tiles.
//   Warp 13 issues the MMAs: P_0 V, S_0 of the next tile, P_1 V, S_1 of the next tile, so that the tensor cores
//   work on one tile while the other's softmax runs.  (Two warps, one a tile, mix the tiles' MMAs and lost 12 %.)
//   Warps 14 and 15 load the tiles' queries: by TMA where the group divides 128 (a box of tokens x heads is
//   128 rows), else by cp.async.
// Bound by the softmax between the products, about 1450 cycles a warpgroup and tile of 128 x 128 beside 1024 of MMAs:
// 8192 tokens of 64 heads of 128, causal, 824 us, 1330 TFLOP/s (72 % of the measured cuBLAS rate).  Short documents
// are bound by the starts and ends of units of about five tiles and by masked tiles, which read S twice (two prompts of 4096
// tokens of 32 heads in documents of 1100: 103 us, capped 152, the special-function unit active 29 % of it).
//
// The work of a batch is one list of key tiles, ordered (sequence, kv head, unit), a unit weighing its tiles
// plus UNIT_COST (its queries' load and output), cut evenly over one persistent CTA per SM: ragged batches,
// causal triangles and few long prompts all end together.  A unit cut by a border leaves partial results
// that a small kernel joins.
//
// e4m3 caches are expanded once into a bf16 copy of the sequences' rows in the workspace (exact: a code times
// a power of two): 256 rows share a tile, so the copy's extra bytes cost less than expanding each tile in
// every unit that reads it would.
#include "gqa_attention.cuh"
#include "tmap.h"

namespace dsv4 {

static __device__ unsigned int g_flags_gp = 0;

namespace gqa {
namespace pre {

constexpr int TILE = 128, UROWS = 256;
constexpr int W_OUT = 8, W_LOAD = 12, W_MMA = 13, W_QUERY = 14, THREADS = 512;
// Registers a thread: 512 x 128 at launch = 256 x 136 (softmax) + 128 x 120 (output) + 128 x 120 (the rest).
constexpr int REGS_SOFTMAX = 136, REGS_OUT = 120, REGS_REST = 120;
constexpr int NSLOT = 4;
// Key tiles that a unit's queries and output weigh in the list (8 x up to 2048 tokens over up to 1000 rows: 270 us at 1, 266 at
// 2, 271 at 3, 279 at 5; 8192 tokens 854, 823, 831, 850).
constexpr int UNIT_COST = 2;
constexpr int FEW_ROWS = 1024;
// Key tiles that are summed into one accumulator.  Adding drops what lies below the accumulator's last bit: the sums lose
// 2^-30 a row or so (outputs 0.13 % low after 2^20 rows, 4.3 % after 2^25), so longer runs are added up in fp32 in the
// workspace.  (A CTA a unit has no place there: calls of more than MAX_UNITS units keep one accumulator.)  Calls whose
// lengths allow such runs take kernels of their own: with that code in the others, 8192 tokens took 834 us for 820, the
// capped documents 162 for 152.
constexpr int MAX_RUN = 2048;
// Units of the evenly cut list: its sums fill the ring's 64 KB.  Above, a CTA takes a whole unit, which costs more (2000
// x 32 tokens over up to 200 rows, e4m3, 1340 us as a list, 1818 so; 1000 x up to 256 over 1000 rows 4.8 ms and 6.7; 32 x up
// to 4096 tokens, bf16, 3.5 and 4.1).
constexpr int MAX_UNITS = 8192;
constexpr float LAZY = 8.f;
// Capped logits lie at most at cap2 = cap log2(e).  A row's reference is put up to 2^CAP_RAISE above its largest logit so
// far, so that cap2 is at most CAP_ROOM above it: then no weight passes 2^20 whatever the rows to come hold (fp32 holds
// 2^20 x rows x values up to 2^107), the largest is at least 2^-60 (its product with values of 2^-40 still has 26
// binary orders of normal numbers below it), and no maximum is needed any more.  It is raised by whole binary orders, so
// that the largest weight is still a power of two and is not rounded (outputs of the capped documents off by 0.0023 with
// a reference at cap2 - 20, 0.0021 so).
constexpr float CAP_ROOM = 20.f, CAP_RAISE = 60.f, CAP_NEAR = CAP_ROOM + 0.5f;
constexpr uint32_t FLAG_TIMEOUT = 4u;
// Longest waits: a tile's 250 ms; those that may span the CTA's whole piece (queries, output, a tile of rows with no work in
// some units) as much and 50 us a key tile that the call's bounds let it hold (a pair of tiles takes 2 us, masked, capped and
// biased 6).
constexpr uint64_t WAIT_NS = 250000000, WAIT_TILE_NS = 50000;

struct Args {
  dsv4_gqa_attention_params p;
  int4* unit;        // [B * tps] of the evenly cut list: first row seen, end of the rows seen, key tiles of tile 0 and 1
                     // (bit 30 of the latter: some page is out of range)
  float4* o_part;    // [2 G][8 groups of 32 rows][D / 4][32 rows]: a warp stores and loads whole lines
  float2* ml_part;   // [2 G][256]
  int4* cut;         // [G]: unit, kv head, last CTA (-1: no unit that begins here goes on), slot here
  uint16_t* bf_k;    // e4m3: the expanded rows [B][kv_heads][kv_pad][D]
  uint16_t* bf_v;
  int kv_pad;
  int tps;           // units a sequence can have
  int G;
  int even;          // 1: the list is cut evenly, 0: a CTA takes a whole unit
  int box;           // cache rows of a TMA box
  int q_tma;         // 1: queries by TMA
  uint64_t piece_ns; // limit of the waits that may span a CTA's piece
};

// ------------------------------------------------------------------------------------------------
// The units' rows (one warp each), and the expansion of e4m3 rows (a CTA per 64 rows and kv head).
// ------------------------------------------------------------------------------------------------
constexpr int PREP_THREADS = 256, EXPAND_ROWS = 64;

// Unit u's rows and tiles (a warp).
__device__ __forceinline__ int4 plan_unit(const Args& a, int u) {
  const dsv4_gqa_attention_params& p = a.p;
  const int lane = threadIdx.x & 31;
  const int b = u / a.tps, tile = u % a.tps, group = p.q_heads / p.kv_heads;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  int4 e = make_int4(0, 0, 0, 0);
  if (!s.ok) {
    if (tile == 0 && lane == 0) atomicOr(&g_flags_gp, FLAG_PAGE);
  } else if ((int64_t)tile * UROWS < (int64_t)s.n * group) {
    int lo = 0x7FFFFFFF, hi[2] = {0, 0};
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r0 = (int64_t)tile * UROWS + i * TILE, r1 = min(r0 + TILE, (int64_t)s.n * group);
      live[i] = r0 < r1;
      if (!live[i]) continue;
      const int t0 = (int)(r0 / group), t1 = (int)((r1 - 1) / group);
      for (int t = t0 + lane; t <= t1; t += 32) {
        const int2 v = visible_rows(p, b, s.t0 + t, s.kv - s.n + t, s.kv);
        if (v.x < v.y) {
          lo = min(lo, v.x);
          hi[i] = max(hi[i], v.y);
        }
      }
      hi[i] = __reduce_max_sync(0xffffffffu, hi[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    if (lo == 0x7FFFFFFF) lo = 0;
    const int start = lo & ~(a.box - 1);
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) n[i] = hi[i] > start ? (hi[i] - start + TILE - 1) / TILE : 0;
    if (live[0]) n[0] = max(n[0], 1);  // (a unit that sees nothing still writes its output)
    const int end = max(hi[0], hi[1]);
    bool bad = false;
    for (int lp = lo / p.page_size + lane; (int64_t)lp * p.page_size < end; lp += 32) {
      const int page = lp < p.max_pages_per_seq ? p.block_table[(int64_t)b * p.max_pages_per_seq + lp] : -1;
      bad |= page < 0 || page >= p.num_pages;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(&g_flags_gp, FLAG_PAGE);
    e = make_int4(lo, end, n[0], n[1] | (bad ? 1 << 30 : 0));
  }
  return e;
}

template <int D>
__device__ __forceinline__ void expand_rows(const Args& a, int item) {
  const dsv4_gqa_attention_params& p = a.p;
  const int blocks = a.kv_pad / EXPAND_ROWS;
  const int blk = item % blocks, u = item / blocks, h = u % p.kv_heads, b = u / p.kv_heads;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  const int r0 = blk * EXPAND_ROWS;
  if (!s.ok || s.n == 0 || r0 >= ((s.kv + TILE - 1) & ~(TILE - 1))) return;
  if (p.window > 0 && r0 + EXPAND_ROWS + TILE <= s.kv - s.n - p.window) return;  // before every token's window
  constexpr int CPR = D / 16;  // 16-byte pieces of a row of codes
  for (int x = threadIdx.x; x < EXPAND_ROWS * CPR; x += PREP_THREADS) {
    const int r = r0 + x / CPR, ch = x % CPR;
    const int lp = r / p.page_size;
    int page = -1;
    if (r < s.kv && lp < p.max_pages_per_seq) page = p.block_table[(int64_t)b * p.max_pages_per_seq + lp];
    const bool in = page >= 0 && page < p.num_pages;
    const int64_t o = (((int64_t)b * p.kv_heads + h) * a.kv_pad + r) * D + ch * 16;
    const int row = r & (p.page_size - 1);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4 w = make_uint4(0, 0, 0, 0);
      float f = 0.f;
      if (in) {
        const uint8_t* src = kv ? reinterpret_cast<const uint8_t*>(p.v_cache) + (int64_t)page * p.v_page_stride +
                                      (int64_t)h * p.v_cache_head_stride + (int64_t)row * p.v_row_stride
                                : reinterpret_cast<const uint8_t*>(p.k_cache) + (int64_t)page * p.k_page_stride +
                                      (int64_t)h * p.k_cache_head_stride + (int64_t)row * p.k_row_stride;
        w = __ldg(reinterpret_cast<const uint4*>(src + ch * 16));
        f = ue8m0_scale((kv ? p.v_exp : p.k_exp)[(int64_t)page * p.kv_heads + h]);
      }
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      uint32_t out[8];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float2 c0 = e4m3x2_to_float2((uint16_t)(ww[y] & 0xFFFFu)), c1 = e4m3x2_to_float2((uint16_t)(ww[y] >> 16));
        out[2 * y] = in ? float2_to_bf16x2_bits(c0.x * f, c0.y * f) : 0u;
        out[2 * y + 1] = in ? float2_to_bf16x2_bits(c1.x * f, c1.y * f) : 0u;
      }
      uint4* dst = reinterpret_cast<uint4*>((kv ? a.bf_v : a.bf_k) + o);
      dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
      dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(PREP_THREADS) prepare_kernel(Args a, int plan_ctas) {
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x < plan_ctas) {
    const int u = blockIdx.x * (PREP_THREADS / 32) + (threadIdx.x >> 5);
    if (u < a.p.B * a.tps) {
      const int4 e = plan_unit(a, u);
      if ((threadIdx.x & 31) == 0) a.unit[u] = e;
    }
  } else {
    expand_rows<D>(a, blockIdx.x - plan_ctas);
  }
}

// ------------------------------------------------------------------------------------------------
// The attention kernel.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(tc::smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(tc::smem_addr(bar))
      : "memory");
}

// Two fp32 values in one register pair: one instruction does both lanes.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct Segment {
  int b, h, tile;      // unit `tile` of sequence b, kv head h
  int lo, end;         // rows seen by the unit: lo .. end - 1
  int start;           // cache row of key tile 0
  int k0, k1, n[2];    // this CTA's key tiles k0 .. k1 - 1; tiles of the two row tiles
  bool bad, whole;     // whole: the segment has all tiles of the unit
  bool add, mine;      // add: to the partial results of the segment before; mine: whole, but for MAX_RUN
  int slot;            // of the unit's partial results in this CTA
  int64_t u0, w;       // the unit's place and weight in the list
  __device__ int count(int i) const { return max(0, min(k1, n[i]) - k0); }
};

// The CTA's segments in order; every warp walks them by itself.
struct Walk {
  const int4* unit;
  const int4* one;  // whole units: the CTA's only entry
  int tps, heads, B, box;
  int b, h, tile;
  int64_t u0, first, last;
  template <bool LONG>
  __device__ __forceinline__ bool next(Segment& g, int& kend) {  // kend: the CTA's tiles of the unit end there (LONG)
    if (LONG && g.k1 < kend) {
      g.k0 = g.k1;
      g.k1 = min(kend, g.k0 + MAX_RUN);
      g.add = true;
      return true;
    }
    while (u0 < last && b < B) {
      const int4 e = one ? *one : unit[(int64_t)b * tps + tile];
      g.n[0] = e.z;
      g.n[1] = e.w & 0x3FFFFFFF;
      g.bad = (e.w >> 30) & 1;
      g.b = b;
      g.h = h;
      g.tile = tile;
      g.lo = e.x;
      g.end = e.y;
      g.start = e.x & ~(box - 1);
      g.u0 = u0;
      const int n = max(g.n[0], g.n[1]);
      g.w = n ? n + UNIT_COST : 0;
      if (++tile == tps || n == 0) {  // (a sequence's units with work come first)
        tile = 0;
        if (++h == heads) {
          h = 0;
          ++b;
        }
      }
      if (n == 0) continue;
      u0 += g.w;
      if (u0 <= first) continue;
      const int64_t x0 = max(first, g.u0) - g.u0, x1 = min(last, u0) - g.u0;
      g.k0 = (int)max((int64_t)0, x0 - UNIT_COST);
      g.k1 = (int)max((int64_t)0, x1 - UNIT_COST);
      if (g.k0 >= g.k1) continue;
      if (LONG) {
        kend = g.k1;
        g.k1 = min(g.k1, g.k0 + MAX_RUN);
        g.mine = g.k0 == 0 && kend == n;
        g.add = false;
      }
      g.whole = g.k0 == 0 && g.k1 == n;
      g.slot = g.u0 <= first ? 0 : 1;
      return true;
    }
    return false;
  }
};

// A warp's walk, in shared memory: lane 0 takes the step, and the state takes no registers from the loops between.
struct WarpWalk {
  Walk w;
  Segment g;
  int have, kend;
  template <bool LONG>
  __device__ __forceinline__ bool next(int lane) {
    __syncwarp();
    if (lane == 0) have = w.next<LONG>(g, kend);
    __syncwarp();
    return have;
  }
};

// x = cap2 tanh(x to_exp / (2 log2 e)) - m for 32 columns, cap2 = cap log2(e), to_exp = 2 log2(e) scale / cap:
// tanh t = 1 - 2 / (1 + e^2t), one reciprocal for two columns; off by at most 2^-20 cap: 2 cap times five roundings of
// the quotient (the reciprocal's counts twice), 10 steps of 2^-24, and 3.3 of the scales' and the exponential's.  With the weight's
// exponential 10 cycles of the special-function unit a warp and column.  (A degree-13 polynomial in packed fp32 was no faster: fp32 pairs issue at half rate.)
__device__ __forceinline__ void cap_logits(uint32_t (&x)[32], float to_exp, float cap2, float m) {
  const float c0 = cap2 - m, c1 = -2.f * cap2;
#pragma unroll
  for (int d = 0; d < 32; d += 2) {
    const float a = 1.f + tc::ex2_approx(fminf(__uint_as_float(x[d]) * to_exp, 60.f));
    const float b = 1.f + tc::ex2_approx(fminf(__uint_as_float(x[d + 1]) * to_exp, 60.f));
    const float r = rcp_approx(a * b);
    x[d] = __float_as_uint(fmaf(r * b, c1, c0));
    x[d + 1] = __float_as_uint(fmaf(r * a, c1, c0));
  }
}

// Weights 2^x of 32 columns: their sums (two chains) and bf16 pairs.
__device__ __forceinline__ void plain_weights(const uint32_t (&x)[32], uint64_t (&sum2)[2], uint32_t (&pk)[16]) {
#pragma unroll
  for (int d = 0; d < 32; d += 2) {
    const float e0 = tc::ex2_approx(__uint_as_float(x[d])), e1 = tc::ex2_approx(__uint_as_float(x[d + 1]));
    sum2[(d >> 1) & 1] = add2(sum2[(d >> 1) & 1], pack2(e0, e1));
    pk[d / 2] = float2_to_bf16x2_bits(e0, e1);
  }
}

struct Smem {
  uint64_t full[NSLOT], empty[NSLOT], vraw, qfull[2], qfree[2], sfull[2], phalf[2], pfull[2], odone[2], ofree[2], stats[2], drain;
  float2 stat[2][TILE];  // a finished tile's (maximum, sum) of each row
  int4 one;              // whole units: the CTA's
  WarpWalk walk[THREADS / 32];
  int64_t first, last, u0;
  int64_t wsum[THREADS / 32];
  int64_t per;
  int b, h, tile;
  uint32_t tmem_base;
  int abort;
};

// One lane of a converged warp.  The MMA warp runs its loop with all lanes and issues under this, so that
// descriptors and barrier addresses stay in uniform registers: issued from a lane == 0 branch, every MMA
// first moved its operands there and 32 of them took 3740 cycles instead of 2048.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// PLAIN: the logits are the scaled scores, the scale positive (its code is half as long, and its loops fetch faster).
// LONG: a CTA may have more than MAX_RUN key tiles of a unit.
template <int D, bool PLAIN, bool LONG>
__global__ void __launch_bounds__(THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap, Args a) {
  constexpr int QT = TILE * D * 2;     // bytes of a query tile, and of a key or value tile
  constexpr int HB = TILE * 128;       // one 64-dim half of it (or all, D = 64)
  constexpr uint32_t COL_O = 256;
  const dsv4_gqa_attention_params& p = a.p;
  extern __shared__ uint8_t raw_mem[];
  uint8_t* mem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_mem) + 1023) & ~uintptr_t(1023));
  uint8_t* q_mem = mem;
  uint8_t* kv_mem = mem + 2 * QT;
  uint8_t* stage_mem = mem + 2 * QT + NSLOT * QT;  // 2 KB an output warp
  Smem* sm = reinterpret_cast<Smem*>(stage_mem + 4 * 2048);
  volatile int* abort = &sm->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    sm->abort = 0;
    for (int i = 0; i < NSLOT; ++i) {
      tc::mbar_init(&sm->full[i], 1);
      tc::mbar_init(&sm->empty[i], 1);
    }
    tc::mbar_init(&sm->vraw, 1);
    tc::mbar_init(&sm->drain, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm->qfull[i], 1);
      tc::mbar_init(&sm->qfree[i], 1);
      tc::mbar_init(&sm->ofree[i], 4);
      tc::mbar_init(&sm->stats[i], 4);
      tc::mbar_init(&sm->sfull[i], 1);
      tc::mbar_init(&sm->phalf[i], 4);
      tc::mbar_init(&sm->pfull[i], 4);
      tc::mbar_init(&sm->odone[i], 1);
    }
    tc::fence_barrier_init();
  }
  if (warp == W_MMA) {
    tc::tmem_alloc(&sm->tmem_base, 512);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---------------- this CTA's piece of the list
  if (a.even) {
    int64_t* pre = reinterpret_cast<int64_t*>(kv_mem);  // inclusive sums of the units' weights
    const int U = p.B * a.tps, per_thread = (U + THREADS - 1) / THREADS;
    const int i0 = min(U, tid * per_thread), i1 = min(U, i0 + per_thread);
    int64_t sum = 0;
    for (int i = i0; i < i1; ++i) {
      const int4 e = a.unit[i];
      const int n = max(e.z, e.w & 0x3FFFFFFF);
      sum += n ? n + UNIT_COST : 0;
      pre[i] = sum;
    }
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm->wsum[warp] = x;
    __syncthreads();
    int64_t off = x - sum, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) off += sm->wsum[w];
      total += sm->wsum[w];
    }
    for (int i = i0; i < i1; ++i) pre[i] += off;
    __syncthreads();
    if (tid == 0) {
      const int64_t all = total * p.kv_heads;
      const int64_t per = max((all + a.G - 1) / a.G, (int64_t)(UNIT_COST + 4));
      const int64_t first = (int64_t)blockIdx.x * per;
      sm->per = per;
      sm->first = first;
      sm->last = min(all, first + per);
      sm->b = p.B;
      if (first < sm->last) {
        int lo = 0, hi = p.B - 1;  // the first b whose units end behind `first`
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (pre[(int64_t)(mid + 1) * a.tps - 1] * p.kv_heads > first) hi = mid;
          else lo = mid + 1;
        }
        const int64_t before = lo ? pre[(int64_t)lo * a.tps - 1] : 0;
        const int64_t W = pre[(int64_t)(lo + 1) * a.tps - 1] - before;
        const int h = (int)((first - before * p.kv_heads) / W);
        const int64_t base = before * p.kv_heads + h * W, x0 = first - base;
        int tl = 0, th = a.tps - 1;  // the first unit that ends behind x0
        while (tl < th) {
          const int mid = (tl + th) >> 1;
          if (pre[(int64_t)lo * a.tps + mid] - before > x0) th = mid;
          else tl = mid + 1;
        }
        sm->b = lo;
        sm->h = h;
        sm->tile = tl;
        sm->u0 = base + (tl ? pre[(int64_t)lo * a.tps + tl - 1] - before : 0);
      }
    }
    if (tid == W_OUT * 32) a.cut[blockIdx.x] = make_int4(0, 0, -1, 0);  // (its writer later)
  } else if (warp == 0) {
    // a whole unit a CTA: units fastest and the last ones (which see most) first, then heads, then sequences
    const int64_t x = blockIdx.x;
    const int tile = a.tps - 1 - (int)(x % a.tps), b = (int)(x / a.tps / p.kv_heads);
    const int4 e = plan_unit(a, b * a.tps + tile);
    if (lane == 0) {
      const int n = max(e.z, e.w & 0x3FFFFFFF);
      sm->tile = tile;
      sm->h = (int)(x / a.tps % p.kv_heads);
      sm->b = b;
      sm->one = e;
      sm->u0 = sm->first = 0;
      sm->last = n ? n + UNIT_COST : 0;
      sm->per = 1;
    }
  }
  tc::fence_proxy_async_smem();  // (the sums lie where key and value tiles will land)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  WarpWalk& ww = sm->walk[warp];
  const Segment& g = ww.g;
  if (lane == 0) {
    Walk& walk = ww.w;
    walk.unit = a.unit;
    walk.one = a.even ? nullptr : &sm->one;
    walk.tps = a.tps;
    walk.heads = p.kv_heads;
    walk.B = p.B;
    walk.box = a.box;
    walk.b = sm->b;
    walk.h = sm->h;
    walk.tile = sm->tile;
    walk.u0 = sm->u0;
    walk.first = sm->first;
    walk.last = sm->last;
    if (LONG) ww.g.k1 = ww.kend = 0;
  }

  if (warp >= W_LOAD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    if (warp == W_LOAD) {
      // ---------------- TMA loads
      int it = 0, armed = 0;  // tiles handed out, tiles armed on their own barrier
      bool raw = false;       // a tile is on its way to vraw
      bool ok = true;
      uint32_t raw_phase = 0;
      if (lane == 0) {
        tc::tma_prefetch_desc(&kmap);
        tc::tma_prefetch_desc(&vmap);
      }
      const int nbox = TILE / a.box;
      const bool expanded = a.bf_k != nullptr;
      while (ok && ww.next<LONG>(lane)) {
        for (int k = g.k0; k < g.k1 && ok; ++k) {
          const int t0 = g.start + k * TILE;
          // box `lane` of the tile: its page (out of range, so that zeros come, where it has none) and row
          int page = expanded ? g.b : (int)max(p.num_pages, (int64_t)1), y = expanded ? t0 : 0;
          if (!expanded && lane < nbox) {
            const int r = t0 + lane * a.box, lp = r / p.page_size;
            if (r < g.end && lp < p.max_pages_per_seq) {
              const int x = p.block_table[(int64_t)g.b * p.max_pages_per_seq + lp];
              if (x >= 0 && x < p.num_pages) page = x;
            }
            y = r & (p.page_size - 1);
          }
          for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
            const int slot = it % NSLOT;
            if (it >= NSLOT) ok = tc::mbar_wait_bounded(&sm->empty[slot], ((it / NSLOT) & 1) ^ 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* dst = kv_mem + slot * QT;
            // value rows that no row of the unit sees may hold anything, and 0 x NaN would reach the output:
            // such a tile lands on a barrier of this warp's, which clears the rows before handing it over
            // (expanded rows from kv_len on are zeros already)
            const bool clear = kv == 1 && (t0 < g.lo || (!expanded && t0 + TILE > g.end));
            uint64_t* bar = clear ? &sm->vraw : &sm->full[slot];
            if (lane == 0) tc::mbar_arrive_expect_tx(bar, QT);
            raw = clear;
            if (!clear) armed = it + 1;
            __syncwarp();
            if (lane < nbox) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(dst + c * HB + lane * a.box * 128, kv ? &vmap : &kmap, c * 64, y, g.h, page, bar);
            }
            if (clear) {
              ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&sm->vraw, raw_phase, abort));
              if (!ok) break;
              raw_phase ^= 1u;
              raw = false;
              armed = it + 1;
              for (int r = lane; r < TILE; r += 32) {
                if (t0 + r >= g.lo && t0 + r < g.end) continue;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                  for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4*>(dst + c * HB + r * 128 + x * 16) = make_uint4(0, 0, 0, 0);
              }
              tc::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&sm->full[slot]);
            }
          }
        }
      }
      if (!ok) {  // gave up: no copy may still be on its way when the CTA ends
        volatile int none = 0;
        for (int x = max(0, armed - NSLOT); x < armed; ++x)
          tc::mbar_wait_bounded(&sm->full[x % NSLOT], (x / NSLOT) & 1, &none, 50000000ull);
        if (raw) tc::mbar_wait_bounded(&sm->vraw, raw_phase, &none, 50000000ull);
      }
    } else if (warp == W_MMA) {
      // ---------------- MMAs
      const uint32_t idesc_s = tc::idesc_bf16_f32(TILE, TILE), idesc_o = tc::idesc_bf16_f32_bmn(TILE, D);
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      const uint64_t qd = tc::sdesc_k_sw128(tc::smem_addr(q_mem)), kd = tc::sdesc_k_sw128(tc::smem_addr(kv_mem));
      const uint64_t vd = tc::sdesc_mn_sw128(tc::smem_addr(kv_mem), HB, 1024);
      int it = 0;
      uint32_t qph[2] = {0, 0}, pph[2] = {0, 0}, oph[2] = {1, 1};  // (ofree: nothing to wait for the first time)
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_bounded(bar, phase, abort));
        tc::tc_fence_after();
      };
      auto wait_full = [&](int x) { wait(&sm->full[x % NSLOT], (x / NSLOT) & 1); };
      auto scores = [&](int i, int x, bool last_one) {
        const uint64_t kb = kd + (uint64_t)((x % NSLOT) * QT >> 4), qb = qd + (uint64_t)(i * QT >> 4);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_bf16(tm + 128 * i, qb + (uint64_t)((c * HB + s * 32) >> 4), kb + (uint64_t)((c * HB + s * 32) >> 4),
                           idesc_s, (c | s) != 0);
          tc::mma_commit(&sm->sfull[i]);
          if (last_one) tc::mma_commit(&sm->qfree[i]);
        }
        __syncwarp();
      };
      auto values = [&](int i, int x, int half, bool more, bool done) {
        const uint64_t vb = vd + (uint64_t)((x % NSLOT) * QT >> 4);
        if (elect_one()) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            tc::mma_bf16_ts(tm + COL_O + D * i, tm + 128 * i + 8 * (4 * half + y),
                            vb + (uint64_t)((4 * half + y) * 2048 >> 4), idesc_o, (more || y) ? 1u : 0u);
          if (done) tc::mma_commit(&sm->odone[i]);
        }
        __syncwarp();
      };
      auto release = [&](int x) {
        if (elect_one()) tc::mma_commit(&sm->empty[x % NSLOT]);
        __syncwarp();
      };
      while (ok && ww.next<LONG>(lane)) {
        const int cnt[2] = {uniform(g.count(0)), uniform(g.count(1))}, n = uniform(g.k1 - g.k0);
        it = uniform(it);
        wait_full(it);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (cnt[i] && ok) {
            wait(&sm->qfull[i], qph[i]);
            qph[i] ^= 1u;
            if (ok) scores(i, it, cnt[i] == 1);
          }
        if (!ok) break;
        release(it);
        for (int k = 0; k < n && ok; ++k, it += 2) {
          wait_full(it + 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (ok && k < cnt[i]) {
              if (k == 0) {
                wait(&sm->ofree[i], oph[i]);  // the output of the unit before has been read
                oph[i] ^= 1u;
              }
              wait(&sm->phalf[i], pph[i]);
              if (!ok) break;
              values(i, it + 1, 0, k > 0, false);
              wait(&sm->pfull[i], pph[i]);
              if (!ok) break;
              values(i, it + 1, 1, true, k == cnt[i] - 1);
              pph[i] ^= 1u;
            }
            if (ok && k + 1 < n) {
              if (i == 0) wait_full(it + 2);
              if (ok && k + 1 < cnt[i]) scores(i, it + 2, k + 2 == cnt[i]);
            }
          }
          if (!ok) break;
          release(it + 1);
          if (k + 1 < n) release(it + 2);
        }
      }
      if (!ok) {  // gave up: no MMA may still run when tensor memory is returned
        volatile int none = 0;
        if (elect_one()) tc::mma_commit(&sm->drain);
        __syncwarp();
        tc::mbar_wait_bounded(&sm->drain, 0, &none, 50000000ull);
      }
    } else if (warp >= W_QUERY) {
      // ---------------- queries of row tile i
      const int i = warp - W_QUERY;
      constexpr int CPR = D / 8, RPI = 32 / CPR;
      const uint32_t group = p.q_heads / p.kv_heads, rpi_q = RPI / group, rpi_r = RPI % group;
      uint32_t fph = 1, armed = 0;  // (qfree: nothing to wait for the first time)
      bool ok = true;
      while (ok && ww.next<LONG>(lane)) {
        if (!g.count(i)) continue;
        const Seq s = sequence(p.q_start, p.kv_len, g.b, p.T, p.max_q_len, p.max_kv_len);
        const uint32_t r0 = (uint32_t)g.tile * UROWS + i * TILE;
        ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&sm->qfree[i], fph, abort, a.piece_ns));
        fph ^= 1u;
        if (!ok) break;
        if (a.q_tma) {
          // (rows of tokens behind the sequence's: another's, or zeros; their output is not written)
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&sm->qfull[i], QT);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(q_mem + i * QT + c * HB, &qmap, c * 64, g.h * (int)group, s.t0 + (int)(r0 / group), 0, &sm->qfull[i]);
          }
          ++armed;
          __syncwarp();
          continue;
        }
        const uint32_t r = r0 + lane / CPR, rows = (uint32_t)s.n * group;
        uint32_t tok = r / group, head = r % group;  // of this lane's first row; then RPI rows on each time
        const int ch = lane % CPR;
        uint8_t* dst = q_mem + i * QT + (ch >> 3) * HB;
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)s.t0 * p.q_token_stride +
                                   (int64_t)g.h * group * p.q_head_stride + 8 * ch;
#pragma unroll 4
        for (int x = 0; x < TILE / RPI; ++x) {
          const int R = x * RPI + lane / CPR;
          const bool in = r + x * RPI < rows;
          tc::cp_async16(dst + R * 128 + (((ch & 7) ^ (R & 7)) << 4),
                         in ? src + (int64_t)tok * p.q_token_stride + (int64_t)head * p.q_head_stride
                            : reinterpret_cast<const __nv_bfloat16*>(p.q),
                         in ? 16u : 0u);
          head += rpi_r;
          tok += rpi_q;
          if (head >= group) {
            head -= group;
            ++tok;
          }
        }
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->qfull[i]);
      }
      if (!ok && armed) {  // gave up: no copy may still be on its way when the CTA ends
        volatile int none = 0;
        tc::mbar_wait_bounded(&sm->qfull[i], (armed - 1) & 1, &none, 50000000ull);
      }
    }
  } else if (warp >= W_OUT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OUT));
    // ---------------- output: warp W_OUT + y writes rows 32 y .. 32 y + 31 of both tiles
    const uint32_t group = p.q_heads / p.kv_heads;
    uint32_t oph[2] = {0, 0};
    bool ok = true;
    while (ok && ww.next<LONG>(lane)) {
      const Seq s = sequence(p.q_start, p.kv_len, g.b, p.T, p.max_q_len, p.max_kv_len);
      const int slot = 2 * blockIdx.x + g.slot;
      const uint32_t n_rows = (uint32_t)s.n * group;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int R = (warp & 3) * 32 + lane, r = i * TILE + R;
        const uint32_t t_o = tmem + ((uint32_t)((warp & 3) * 32) << 16) + COL_O + D * i;
        const uint32_t ru = (uint32_t)g.tile * UROWS + r;
        const bool live = ru < n_rows;
        const int head = g.h * (int)group + (int)(ru % group);
        const int64_t row = (int64_t)(s.t0 + (int)(ru / group)) * p.q_heads + head;
        const int cnt = g.count(i);
        float m = -INFINITY, l = 0.f;
        if (cnt) {
          ok = tc::mbar_wait_bounded(&sm->stats[i], oph[i], abort, a.piece_ns) &&
               tc::mbar_wait_bounded(&sm->odone[i], oph[i], abort);
          ok = __all_sync(0xffffffffu, ok);
          oph[i] ^= 1u;
          if (!ok) break;
          tc::tc_fence_after();
          const float2 ml = sm->stat[i][R];
          m = ml.x;
          l = ml.y;
        }
        const bool some = m > -INFINITY;  // (a row that saw nothing: what O holds does not matter)
        float f = 1.f, f0 = 0.f;          // f0: the factor of the partial results so far
        if (g.whole) {
          if (live) f = finish_scale(p, row, head, m, l, true);
        } else {
          float2* ml = a.ml_part + (int64_t)slot * UROWS + r;
          if (LONG && g.add) {
            const float2 x = *ml;
            const float mn = fmaxf(m, x.x);
            f = some ? tc::ex2_approx(m - mn) : 0.f;
            f0 = x.x > -INFINITY ? tc::ex2_approx(x.x - mn) : 0.f;
            l = l * f + x.y * f0;
            m = mn;
          }
          *ml = make_float2(m, l);
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (cnt) {
            tc::tmem_ld32_nowait(t_o + c, o);
            tc::tmem_wait_ld_regs<32>(o);
          }
#pragma unroll
          for (int d = 0; d < 32; ++d) o[d] = some ? __float_as_uint(__uint_as_float(o[d]) * f) : 0u;
          if (!g.whole) {
            float4* dst = a.o_part + (((int64_t)slot * 8 + i * 4 + (warp & 3)) * (D / 4) + c / 4) * 32 + lane;
#pragma unroll
            for (int d = 0; d < 32; d += 4) {
              float4 v = make_float4(__uint_as_float(o[d]), __uint_as_float(o[d + 1]), __uint_as_float(o[d + 2]),
                                     __uint_as_float(o[d + 3]));
              if (LONG && g.add) {
                const float4 x = dst[d * 8];
                v.x = fmaf(x.x, f0, v.x);
                v.y = fmaf(x.y, f0, v.y);
                v.z = fmaf(x.z, f0, v.z);
                v.w = fmaf(x.w, f0, v.w);
              }
              dst[d * 8] = v;
            }
          } else if (p.out_dtype == DSV4_F32) {
            if (live) {
#pragma unroll
              for (int d = 0; d < 32; d += 4)
                *reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.out) + row * D + c + d) =
                    make_uint4(o[d], o[d + 1], o[d + 2], o[d + 3]);
            }
          } else {
            // 32 dims of the warp's 32 rows turn in shared memory (16-byte pieces, exchanged by row), so that a store
            // writes whole sectors of 8 rows
            uint4* stage = reinterpret_cast<uint4*>(stage_mem) + (warp & 3) * 128;
            __syncwarp();
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[y] = float2_to_bf16x2_bits(__uint_as_float(o[8 * d + 2 * y]), __uint_as_float(o[8 * d + 2 * y + 1]));
              stage[lane * 4 + (d ^ ((lane >> 1) & 3))] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int rr = x * 8 + (lane >> 2), d = lane & 3;
              const uint4 w = stage[rr * 4 + (d ^ ((rr >> 1) & 3))];
              const int64_t ro = __shfl_sync(0xffffffffu, row, rr);
              if ((uint32_t)g.tile * UROWS + i * TILE + (warp & 3) * 32 + rr < n_rows)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + ro * D + c + 8 * d) = w;
            }
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (cnt && lane == 0) tc::mbar_arrive(&sm->ofree[i]);
        if (LONG && g.mine && g.add && g.k1 == ww.kend && live) {  // the sums of a unit of several segments are complete
          const float y = finish_scale(p, row, head, m, l, true);
          const float4* src = a.o_part + ((int64_t)slot * 8 + i * 4 + (warp & 3)) * (D / 4) * 32 + lane;
#pragma unroll 1
          for (int d4 = 0; d4 < D / 4; ++d4) {
            const float4 x = src[d4 * 32];
            store4<D>(p, row, d4, make_float4(x.x * y, x.y * y, x.z * y, x.w * y));
          }
        }
      }
      if (warp == W_OUT && lane == 0 && !(LONG ? g.mine : g.whole) && g.k0 == 0)
        // the unit's first piece: it goes on up to the CTA of its last tile
        a.cut[blockIdx.x] = make_int4(g.b * a.tps + g.tile, g.h, (int)((g.u0 + g.w - 1) / sm->per), g.slot);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ---------------- softmax: warpgroup i owns row tile i, a thread a row
    const int i = warp >> 2, R = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + 128 * i, t_o = lanes + COL_O + D * i;
    const uint32_t group = p.q_heads / p.kv_heads;
    constexpr bool plain = PLAIN;
    const bool capped = !PLAIN && p.softcap > 0.f && p.slopes == nullptr;
    const float cl = p.softmax_scale * LOG2E, cap2 = p.softcap * LOG2E;
    const float to_exp = p.softcap > 0.f ? 2.f * LOG2E * p.softmax_scale / p.softcap : 0.f;
    uint32_t sph = 0, fph = 1;  // (ofree: nothing to wait for the first time)
    bool ok = true;
    while (ok && ww.next<LONG>(lane)) {
      const int cnt = g.count(i);
      if (!cnt) continue;
      const Seq s = sequence(p.q_start, p.kv_len, g.b, p.T, p.max_q_len, p.max_kv_len);
      const uint32_t ru = (uint32_t)g.tile * UROWS + i * TILE + R;
      const bool live = ru < (uint32_t)s.n * group;
      const int tok = (int)(ru / group), head = g.h * (int)group + (int)(ru % group), pos = s.kv - s.n + tok;
      int2 vis = make_int2(0, 0);
      float slope = 0.f;
      if (live) {
        vis = visible_rows(p, g.b, s.t0 + tok, pos, s.kv);
        if (!PLAIN && p.slopes) slope = p.slopes[head] * LOG2E;
      }
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < cnt; ++k) {
        ok = tc::mbar_wait_bounded(&sm->sfull[i], sph, abort, a.piece_ns);
        sph ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::tc_fence_after();
        const int t0 = g.start + (g.k0 + k) * TILE;
        const bool inside = !live || (t0 >= vis.x && t0 + TILE <= vis.y);
        // The row's maximum: S is read from tensor memory a first time, 32 columns ahead of the work on 32.
        // Where something has to be done to the logits, they go back in log2 units and the maximum is theirs.
        uint32_t xa[32], xb[32];
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float mul = cl;
        const bool all = __all_sync(0xffffffffu, inside && !g.bad);
        if (capped && all && __all_sync(0xffffffffu, cap2 - m <= CAP_NEAR)) {
          // No maximum is needed, and the tile is read once.  (Rolled: this code is long, and instruction fetch counts.)
          uint64_t sum2[2] = {0, 0};
          tc::tmem_ld32_nowait(t_s, xa);
          tc::tmem_wait_ld_regs<32>(xa);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (c < 3) tc::tmem_ld32_nowait(t_s + 32 * (c + 1), xb);
            uint32_t pk[16];
            cap_logits(xa, to_exp, cap2, m);
            plain_weights(xa, sum2, pk);
            if (c < 3) tc::tmem_wait_ld_regs<32>(xb);  // (P lies over columns that have been read)
            tc::tmem_st16(t_s + 16 * c, pk);
#pragma unroll
            for (int d = 0; d < 32; ++d) xa[d] = xb[d];
            if (c & 1) {
              tc::tmem_wait_st();
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(c == 1 ? &sm->phalf[i] : &sm->pfull[i]);
            }
          }
          const float2 sums = unpack2(add2(sum2[0], sum2[1]));
          l += sums.x + sums.y;
          continue;
        }
        if (plain && all) {
          tc::tmem_ld32_nowait(t_s, xa);
          tc::tmem_wait_ld_regs<32>(xa);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t* cur = c & 1 ? xb : xa;
            uint32_t* nxt = c & 1 ? xa : xb;
            if (c < 3) tc::tmem_ld32_nowait(t_s + 32 * (c + 1), nxt);
#pragma unroll
            for (int d = 0; d < 32; ++d) tops[d & 3] = fmaxf(tops[d & 3], __uint_as_float(cur[d]));
            if (c < 3) tc::tmem_wait_ld_regs<32>(nxt);
          }
        } else {
          if (!plain) mul = 1.f;
#pragma unroll 1
          for (int c = 0; c < TILE; c += 32) {
            tc::tmem_ld32_nowait(t_s + c, xa);
            int lo = max(0, vis.x - t0 - c), hi = min(32, vis.y - t0 - c);
            uint32_t see = 0;  // bit d: the row sees column c + d
            if (hi > lo) see = (0xFFFFFFFFu >> (32 - (hi - lo))) << lo;
            if (g.bad) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int j = t0 + c + 16 * y, lp = j / p.page_size;
                const int page = j < g.end && lp < p.max_pages_per_seq
                                     ? p.block_table[(int64_t)g.b * p.max_pages_per_seq + lp] : -1;
                if (page < 0 || page >= p.num_pages) see &= ~(0xFFFFu << (16 * y));
              }
            }
            tc::tmem_wait_ld_regs<32>(xa);
            if (!PLAIN && p.softcap > 0.f) {
              cap_logits(xa, to_exp, cap2, 0.f);
            } else if (!plain) {
#pragma unroll
              for (int d = 0; d < 32; ++d) xa[d] = __float_as_uint(__uint_as_float(xa[d]) * cl);
            }
            if (!PLAIN && p.slopes) {
              const float far = (float)(pos - t0 - c);
#pragma unroll
              for (int d = 0; d < 32; ++d)
                xa[d] = __float_as_uint(fmaf(-slope, fabsf(far - (float)d), __uint_as_float(xa[d])));
            }
            if (!all) {
#pragma unroll
              for (int d = 0; d < 32; ++d)
                if (!((see >> d) & 1u)) xa[d] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int d = 0; d < 32; ++d) tops[d & 3] = fmaxf(tops[d & 3], __uint_as_float(xa[d]));
            tc::tmem_st32(t_s + c, xa);
          }
          tc::tmem_wait_st();
        }
        const float top = mul * fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        const float want = capped ? top + fminf(fmaxf(ceilf(cap2 - CAP_ROOM - top), 0.f), CAP_RAISE) : top;
        const bool move = capped && cap2 - m > CAP_NEAR ? want > m : top > m + LAZY;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? want : m;
          const float f = m == -INFINITY ? 0.f : tc::ex2_approx(m - mn);
          m = mn;
          l *= f;
          if (k > 0) {  // (the scores' commit also covers the product of the tile before)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::tmem_ld32_nowait(t_o + c, o);
              tc::tmem_wait_ld_regs<32>(o);
#pragma unroll
              for (int d = 0; d < 32; ++d) o[d] = __float_as_uint(__uint_as_float(o[d]) * f);
              tc::tmem_st32(t_o + c, o);
            }
          }
        }
        tc::tmem_ld32_nowait(t_s, xa);
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t mul2 = pack2(mul, mul), ref2 = pack2(-mm, -mm);
        uint64_t sum2[2] = {0, 0};
        tc::tmem_wait_ld_regs<32>(xa);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t* cur = c & 1 ? xb : xa;
          uint32_t* nxt = c & 1 ? xa : xb;
          if (c < 3) tc::tmem_ld32_nowait(t_s + 32 * (c + 1), nxt);
          uint32_t pk[16];
#pragma unroll
          for (int d = 0; d < 32; d += 2) {
            const float2 z = unpack2(fma2(pack2u(cur[d], cur[d + 1]), mul2, ref2));
            const float e0 = tc::ex2_approx(z.x), e1 = tc::ex2_approx(z.y);
            sum2[(d >> 1) & 1] = add2(sum2[(d >> 1) & 1], pack2(e0, e1));
            pk[d / 2] = float2_to_bf16x2_bits(e0, e1);
          }
          if (c < 3) tc::tmem_wait_ld_regs<32>(nxt);  // (P lies over columns that have been read)
          tc::tmem_st16(t_s + 16 * c, pk);
          if (c == 1) {  // the product can start on the first half
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm->phalf[i]);
          }
        }
        const float2 sums = unpack2(add2(sum2[0], sum2[1]));
        l += sums.x + sums.y;
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->pfull[i]);
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&sm->ofree[i], fph, abort));  // the stats before have been read
      fph ^= 1u;
      if (!ok) break;
      sm->stat[i][R] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->stats[i]);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm->abort) atomicOr(&g_flags_gp, FLAG_TIMEOUT);
  if (warp == W_MMA) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The units that a border between CTAs cuts: CTA (c, y) joins rows 32 y .. 32 y + 31 of the one that begins in
// CTA c; a lane has a row, a warp D / 8 of its dims.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const dsv4_gqa_attention_params& p = a.p;
  const int4 cut = a.cut[blockIdx.x];
  if (cut.z < 0) return;
  const int b = cut.x / a.tps, tile = cut.x % a.tps, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t group = p.q_heads / p.kv_heads;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  const int parts = cut.z - (int)blockIdx.x + 1, rr = blockIdx.y * 32 + lane;
  const uint32_t r = (uint32_t)tile * UROWS + rr;
  if (r >= (uint32_t)s.n * group) return;
  constexpr int E = D / 32;  // float4s of a warp's dims
  auto place = [&](int i) { return (int64_t)2 * (blockIdx.x + i) + (i == 0 ? cut.w : 0); };
  float m = -INFINITY, l = 0.f;
  float4 acc[E];
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < parts; ++i) m = fmaxf(m, a.ml_part[place(i) * UROWS + rr].x);
#pragma unroll 2
  for (int i = 0; i < parts; ++i) {
    const float2 ml = a.ml_part[place(i) * UROWS + rr];
    const float f = ml.x > -INFINITY ? tc::ex2_approx(ml.x - m) : 0.f;  // (its sums are zeros then)
    l += ml.y * f;
    const float4* src = a.o_part + ((place(i) * 8 + blockIdx.y) * (D / 4) + warp * E) * 32 + lane;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float4 v = src[k * 32];
      acc[k].x = fmaf(v.x, f, acc[k].x);
      acc[k].y = fmaf(v.y, f, acc[k].y);
      acc[k].z = fmaf(v.z, f, acc[k].z);
      acc[k].w = fmaf(v.w, f, acc[k].w);
    }
  }
  const int head = cut.y * (int)group + (int)(r % group);
  const int64_t row = (int64_t)(s.t0 + (int)(r / group)) * p.q_heads + head;
  const float f = finish_scale(p, row, head, m, l, warp == 0);
#pragma unroll
  for (int k = 0; k < E; ++k)
    store4<D>(p, row, warp * E + k, make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f));
}

struct Plan {
  int tps, G, even, kv_pad;
  size_t unit, part, ml, cut, k, v, total;
};

static Plan plan(const dsv4_gqa_attention_params& p) {
  Plan L;
  const int64_t max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  L.tps = (int)((max_n * (p.q_heads / p.kv_heads) + UROWS - 1) / UROWS);
  const int64_t units = (int64_t)p.B * L.tps;
  L.G = num_sms();
  // A CTA a unit where that fills the device at most twice with few key tiles each: it needs no list, no join and, for
  // bf16 caches, no kernel before it (bf16, 32 heads, 8 kv heads: one prompt of 512 tokens 17 us, 28 as a list; 4 x 256
  // over 700 rows 26 and 39; up to 4096 rows and four times the device: 256 tokens over 2000 rows 40 for 32, 8 x 512
  // over 400 rows 83 for 78).  And beyond MAX_UNITS.
  const bool few = units * p.kv_heads <= 2 * L.G && p.max_kv_len <= FEW_ROWS;
  L.even = units <= MAX_UNITS && !few;
  const size_t slots = L.even ? 2 * (size_t)L.G : 0;
  L.kv_pad = p.cache_dtype == DSV4_E4M3_PAGE ? (p.max_kv_len + TILE - 1) / TILE * TILE : 0;
  const size_t rows = (size_t)p.B * p.kv_heads * L.kv_pad * p.head_dim * 2;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = align_up(at + bytes, 256);
    return x;
  };
  L.unit = take(L.even ? (size_t)units * 16 : 0);
  L.part = take(slots * UROWS * p.head_dim * 4);
  L.ml = take(slots * UROWS * 8);
  L.cut = take((size_t)L.G * 16);
  L.k = take(rows);
  L.v = take(rows);
  L.total = at;
  return L;
}

template <int D>
static cudaError_t launch(const dsv4_gqa_attention_params& p, cudaStream_t s) {
  const Plan L = plan(p);
  uint8_t* ws = reinterpret_cast<uint8_t*>(p.workspace);
  Args a;
  a.p = p;
  a.unit = reinterpret_cast<int4*>(ws + L.unit);
  a.o_part = reinterpret_cast<float4*>(ws + L.part);
  a.ml_part = reinterpret_cast<float2*>(ws + L.ml);
  a.cut = reinterpret_cast<int4*>(ws + L.cut);
  const bool e4m3 = p.cache_dtype == DSV4_E4M3_PAGE && L.kv_pad > 0;
  a.bf_k = e4m3 ? reinterpret_cast<uint16_t*>(ws + L.k) : nullptr;
  a.bf_v = e4m3 ? reinterpret_cast<uint16_t*>(ws + L.v) : nullptr;
  a.kv_pad = L.kv_pad;
  a.tps = L.tps;
  a.G = L.G;
  a.even = L.even;
  a.box = e4m3 || p.page_size > TILE ? TILE : p.page_size;
  const int64_t units = (int64_t)p.B * L.tps;
  const int64_t plan_ctas = L.even ? (units + PREP_THREADS / 32 - 1) / (PREP_THREADS / 32) : 0;
  const int64_t expand = e4m3 ? (int64_t)p.B * p.kv_heads * (L.kv_pad / EXPAND_ROWS) : 0;
  const int64_t ctas = L.even ? L.G : units * p.kv_heads;
  const int64_t weight = p.max_kv_len / TILE + 2 + UNIT_COST;  // of a unit, at most
  a.piece_ns = WAIT_NS + WAIT_TILE_NS * (uint64_t)(L.even ? units * p.kv_heads * weight / L.G + weight : weight);
  if (plan_ctas + expand > 0x7FFFFFFF || ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  CUtensorMap kmap, vmap;
  cudaError_t e;
  if (e4m3) {
    const int64_t row = D * 2, head = row * L.kv_pad, seq = head * p.kv_heads;
    e = make_tmap_4d_bf16(&kmap, a.bf_k, D, L.kv_pad, p.kv_heads, p.B, row, head, seq, 64, TILE, 1);
    if (e == cudaSuccess) e = make_tmap_4d_bf16(&vmap, a.bf_v, D, L.kv_pad, p.kv_heads, p.B, row, head, seq, 64, TILE, 1);
  } else {
    const uint64_t pages = p.num_pages > 0 ? p.num_pages : 1;
    e = make_tmap_4d_bf16(&kmap, p.k_cache, D, p.page_size, p.kv_heads, pages, 2 * p.k_row_stride, 2 * p.k_cache_head_stride,
                          2 * p.k_page_stride, 64, a.box, 1);
    if (e == cudaSuccess)
      e = make_tmap_4d_bf16(&vmap, p.v_cache, D, p.page_size, p.kv_heads, pages, 2 * p.v_row_stride,
                            2 * p.v_cache_head_stride, 2 * p.v_page_stride, 64, a.box, 1);
  }
  if (e != cudaSuccess) return e;
  // queries: a box of TILE / group tokens x the group's heads; strides TMA can take
  const int group = p.q_heads / p.kv_heads;
  CUtensorMap qmap = kmap;
  const int64_t ts = 2 * p.q_token_stride, hs = 2 * p.q_head_stride;
  a.q_tma = TILE % group == 0 && ts > 0 && hs > 0 && ts < (1LL << 40) && hs < (1LL << 40);
  if (a.q_tma) {
    e = make_tmap_4d_bf16(&qmap, p.q, D, p.q_heads, p.T, 1, hs, ts, ts, 64, group, TILE / group);
    if (e != cudaSuccess) a.q_tma = 0;
  }
  const int smem = (2 + NSLOT) * TILE * D * 2 + 4 * 2048 + (int)sizeof(Smem) + 1024;
  const bool plain = p.softcap == 0.f && p.slopes == nullptr && p.softmax_scale > 0.f;
  const bool lng = L.even && p.max_kv_len > MAX_RUN * TILE;
  const auto kernel = plain ? (lng ? prefill_kernel<D, true, true> : prefill_kernel<D, true, false>)
                            : (lng ? prefill_kernel<D, false, true> : prefill_kernel<D, false, false>);
  e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  if (plan_ctas + expand > 0) {
    e = launch_pdl(prepare_kernel<D>, dim3((unsigned)(plan_ctas + expand)), dim3(PREP_THREADS), 0, s, true, a, (int)plan_ctas);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(THREADS), smem, s, true, kmap, vmap, qmap, a);
  if (e != cudaSuccess || !L.even) return e;
  return launch_pdl(join_kernel<D>, dim3(L.G, UROWS / 32), dim3(256), 0, s, true, a);
}

}  // namespace pre

size_t prefill_workspace(const dsv4_gqa_attention_params& p) { return pre::plan(p).total; }

cudaError_t launch_prefill(const dsv4_gqa_attention_params& p, cudaStream_t s) {
  return p.head_dim == 128 ? pre::launch<128>(p, s) : pre::launch<64>(p, s);
}

}  // namespace gqa

cudaError_t read_flags_gqa_prefill(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_gp, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_gp, &z, sizeof(z));
}

}  // namespace dsv4
