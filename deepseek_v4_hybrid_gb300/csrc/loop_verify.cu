// Verification of drafted tokens.
//
// A cluster of CTAs takes a sequence, each CTA the same slice of the vocabulary of every row.  Rows are taken in groups:
// the warps go over the slices of a group's rows once, with a reference and the sum of e^(z - reference) of a
// softmax (in 32-bit floats), the CTAs exchange these through distributed shared memory, and every CTA
// finds by itself how far the drafted tokens stand.  The row where they end is read once more, from the L2 cache,
// for the race argmax r(x) / noise(x), whose winners are exchanged the same way.  Rows behind that group are not read.
//
// Two CTAs of 256 threads an SM with six groups of copies on their way each (512 threads, four groups: 256 x 5 rows of
// 131072 logits 171 us for 133, 64 x 4 rows 44 for 36; three CTAs with four groups 173 and 43).  Large batches are bound
// by HBM: 256 x 5 rows of 131072 bf16 logits of both models 133 us, of which the 651 MB that the drafts that stand make
// it read take 96 at the copy rate.  Smaller ones by a chain of phases, each waiting for the one before: launch and first
// loads (2 us), rows, exchange and decision (3 us), race, exchange; 2 x 4 rows of 32000 fp32 logits 11.7 us, 64 x 4 rows of
// 131072 bf16 logits with fp32 probabilities of the draft 36.4 us (103 MB), 200 x up to 3 rows of 100003 45.5 us.
// Code that runs once a sequence waits for its instructions to be fetched: parts that would be inlined twice are loops.
// Exponents are taken of differences from a logit, in two instructions for one fused product against an integer, which
// leaves no range that logits or low temperatures could leave.
#include <cooperative_groups.h>

#include "loop_common.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace dsv4 {

static __device__ unsigned int g_flags_vf = 0;

namespace loop {

namespace cg = cooperative_groups;

constexpr int MAX_CLUSTER = 8, MAX_ROWS = 8;  // rows of a group
constexpr double LOG2E = 1.4426950408889634;  // in two floats:
constexpr float LOG2E_HI = (float)LOG2E, LOG2E_LO = (float)(LOG2E - (double)LOG2E_HI), LN2F = 0.69314718055994531f;
constexpr float MAX_F32 = 3.4028234663852886e38f, MAX_BF16 = 3.3895313892515355e38f;
constexpr int NOWHERE = 0x7FFFFFFF;

constexpr int U = 4;  // vectors of a block of a lane (scan), 32 vectors apart

// Sums of a part of a row of logits, weights 2^((z - m) c) against the reference m, one of the row's logits (-inf: the part
// leaves nothing): `top` of the lane's block that weighs most, s of all other elements.  A token of a probability p over a half
// lies in that block, and -log p = log1p(rest / its weight): rest, the others' sum, would be lost in the roundings of a sum that
// has the token in it.  `where` is the block's first element, and its vectors (0: that element alone) from bit 24 on.
// For greedy sequences m is the maximum, and idx its first index.
struct Stat {
  float m, s, top;
  int where, idx;
};
constexpr Stat NOTHING = {-INFINITY, 0.f, 0.f, 0, NOWHERE};

__device__ __forceinline__ void merge(Stat& a, Stat b, float c) {
  if (b.m == -INFINITY) return;
  if (a.m == -INFINITY) {
    a = b;
    return;
  }
  const float f = tc::ex2_approx(-fabsf(a.m - b.m) * c);
  if (b.m > a.m) {
    a.s *= f, a.top *= f, a.m = b.m, a.idx = b.idx;
  } else {
    b.s *= f, b.top *= f;
    if (b.m == a.m) a.idx = min(a.idx, b.idx);
  }
  a.s += b.s + fminf(a.top, b.top);
  if (b.top > a.top) a.top = b.top, a.where = b.where;
}

// A logit as it counts: NaN as -inf, +inf as the type's largest value.
__device__ __forceinline__ float largest(bool f32) { return f32 ? MAX_F32 : MAX_BF16; }
__device__ __forceinline__ float logit(float x, bool f32) { return fminf(fmaxf(x, -INFINITY), largest(f32)); }
// A probability: NaN and negative ones as 0.
__device__ __forceinline__ float prob(float x) { return fminf(fmaxf(x, 0.f), MAX_F32); }

template <bool F32>
__device__ __forceinline__ float element(const void* base, int64_t i) {
  return F32 ? reinterpret_cast<const float*>(base)[i]
             : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[i] << 16);
}
__device__ __forceinline__ float element(const void* base, int64_t i, bool f32) {
  return f32 ? element<true>(base, i) : element<false>(base, i);
}
__device__ __forceinline__ const void* at(const void* base, int64_t i, bool f32) {
  return reinterpret_cast<const uint8_t*>(base) + i * (f32 ? 4 : 2);
}

// Two floats in one register pair, for the packed instructions.
__device__ __forceinline__ uint64_t pack(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 16 bytes of a row.
template <bool F32>
struct Vec {
  static constexpr int E = F32 ? 4 : 8;
  uint32_t w[4];
  __device__ __forceinline__ void set(const uint4& r) { w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w; }
  __device__ __forceinline__ float get(int i) const {
    if (F32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};
template <bool F32>
constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;  // elements of -inf

// The largest of the elements (NaN is passed over).
template <bool F32, int N>
__device__ __forceinline__ float top_of(const Vec<F32> (&v)[N]) {
  if (F32) {
    float top = v[0].get(0);
#pragma unroll
    for (int i = 1; i < N * 4; ++i) top = fmaxf(top, v[i / 4].get(i % 4));
    return top;
  }
  __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&v[0].w[0]);
#pragma unroll
  for (int i = 1; i < N * 4; ++i) y = __hmax2(y, *reinterpret_cast<const __nv_bfloat162*>(&v[i / 4].w[i % 4]));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&y);
  return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Order-preserving map of floats (no NaN) to integers and back.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b < 0 ? b ^ 0x7FFFFFFF : b;
}
__device__ __forceinline__ float from_ordered(int k) { return __int_as_float(k < 0 ? k ^ 0x7FFFFFFF : k); }
__device__ __forceinline__ float warp_top(float x) { return from_ordered(__reduce_max_sync(0xffffffffu, ordered(x))); }

// Each thread streams its vectors through a ring of its own in shared memory: groups of asynchronous 16-byte copies,
// all but one of them ahead of the one in use.  Nobody else reads them, so no barrier is needed.

// The running numbers of a warp over a row: the reference m, one of its logits, and the lane's sums of 2^((z - m) c): `top` of
// the block of 32 elements (16 of fp32) that weighs most, begun at vector `at`, and s of the others.
// Greedy sequences keep m at the maximum and each lane's first index of it; the others change it only when the sum of
// a block says that one lies above it by a binary order or two, which spares the search.  (An exponent's
// argument y is off by |y| 2^-22, so the elements that make up the sum should have small ones.)
// Elements are taken as they are: NaN and +inf make the sum NaN, and the part is then done again by the careful form.
constexpr float FAR = 64.f;
constexpr int FRONT = -1, BACK = -2;  // blocks of one element a lane, before and behind the whole vectors

struct Run {
  float m, s, top;
  int at, idx;
};

template <bool F32, int N>
__device__ __forceinline__ float weights(const Vec<F32> (&v)[N], float c, float m) {
  constexpr int E = Vec<F32>::E;
  const uint64_t c2 = pack(c, c), m2 = pack(-m, -m);
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < N * E; i += 2) {
    const uint64_t y = mul2(add2(pack(v[i / E].get(i % E), v[i / E].get(i % E + 1)), m2), c2);
    sum = add2(sum, pack(tc::ex2_approx(low(y)), tc::ex2_approx(high(y))));
  }
  return low(sum) + high(sum);
}

template <bool F32, bool GREEDY, int N, typename I>
__device__ __forceinline__ void add(Run& st, const Vec<F32> (&v)[N], float c, int block, I index) {
  constexpr int E = Vec<F32>::E;
  bool look = GREEDY || st.m == -INFINITY;
  while (true) {  // (a loop, so that each part of the code is there once: what runs once a row waits for its instructions)
    if (look) {
      const float top = top_of<F32, N>(v);
      if (__any_sync(0xffffffffu, top > st.m)) {
        const float m = warp_top(fmaxf(top, st.m));
        if (st.m > -INFINITY) {
          const float f = tc::ex2_approx((st.m - m) * c);
          st.s *= f, st.top *= f;
        }
        st.m = m;
        if (GREEDY) {
          st.idx = NOWHERE;
          if (top == m) {
#pragma unroll
            for (int i = N * E - 1; i >= 0; --i)
              if (v[i / E].get(i % E) == m) st.idx = index(i);
          }
        }
      }
    }
    const float sum = weights<F32, N>(v, c, st.m == -INFINITY ? 0.f : st.m);
    if (look || !__any_sync(0xffffffffu, sum > FAR)) {
      const bool higher = sum > st.top;
      st.s += higher ? st.top : sum;
      if (higher) st.top = sum, st.at = block;
      return;
    }
    look = true;
  }
}

// The careful form: one element, as it counts; m is the maximum, and its first place the block of its own that is left out of s.
__device__ __forceinline__ void add_careful(Stat& st, float z, int i, float c) {
  if (z == -INFINITY) return;
  if (z > st.m) {
    st.s = st.m == -INFINITY ? 0.f : (st.s + 1.f) * tc::ex2_approx((st.m - z) * c);
    st.m = z, st.idx = i;
  } else {
    st.s += tc::ex2_approx((z - st.m) * c);
  }
}

// Elements [lo, hi) of a row of logits: warp `share` of `shares` takes its part, blocks of U * 32 vectors, and returns its
// numbers in every lane.
template <int NT, int DEPTH, bool F32, bool GREEDY>
__device__ __noinline__ Stat scan_row(const void* row, int lo, int hi, int share, int shares, float c, uint4* ring) {
  constexpr int E = Vec<F32>::E, BLOCK = U * 32;
  const int lane = threadIdx.x & 31;
  const uintptr_t a = reinterpret_cast<uintptr_t>(at(row, lo, F32));
  const int head = min(hi - lo, (int)((16 - (a & 15)) & 15) / (F32 ? 4 : 2));  // elements before the first whole 16 bytes
  const int from = lo + head, vecs = (hi - from) / E, step = BLOCK * shares;
  const uint4* v = reinterpret_cast<const uint4*>(at(row, from, F32)) + lane;
  uint4* mine = ring + threadIdx.x;
  const auto fetch = [&](int j0, int group) {  // the block from vector j0 on
    uint4* to = mine + group * (U * NT);
    if (j0 + BLOCK <= vecs) {
#pragma unroll
      for (int u = 0; u < U; ++u) tc::cp_async16(to + u * NT, v + j0 + u * 32, 16);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u * 32 + lane < vecs) tc::cp_async16(to + u * NT, v + j0 + u * 32, 16);
    }
    tc::cp_async_commit();
  };
  int j0 = share * BLOCK, ahead = j0, to = 0, use = 0;
#pragma unroll
  for (int g = 0; g < DEPTH - 1; ++g, ahead += step, ++to) fetch(ahead, to);
  Run st = {-INFINITY, 0.f, 0.f, FRONT, NOWHERE};
  const auto one = [&](int i, bool there, int block) {
    Vec<F32> z[1];
    z[0].set(make_uint4(NONE<F32>, NONE<F32>, NONE<F32>, NONE<F32>));
    if (there) z[0].w[0] = F32 ? reinterpret_cast<const uint32_t*>(row)[i] : 0xFF800000u | reinterpret_cast<const uint16_t*>(row)[i];
    add<F32, GREEDY, 1>(st, z, c, block, [&](int) { return i; });
  };
  if (share == 0 && head > 0) one(lo + lane, lane < head, FRONT);
  for (; j0 < vecs; j0 += step, ahead += step) {
    fetch(ahead, to);
    to = to == DEPTH - 1 ? 0 : to + 1;
    tc::cp_async_wait<DEPTH - 1>();
    const uint4* block = mine + use * (U * NT);
    use = use == DEPTH - 1 ? 0 : use + 1;
    Vec<F32> z[U];
    if (j0 + BLOCK <= vecs) {
#pragma unroll
      for (int u = 0; u < U; ++u) z[u].set(block[u * NT]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        z[u].set(make_uint4(NONE<F32>, NONE<F32>, NONE<F32>, NONE<F32>));
        if (j0 + u * 32 + lane < vecs) z[u].set(block[u * NT]);
      }
    }
    add<F32, GREEDY, U>(st, z, c, j0, [&](int i) { return from + (j0 + i / E * 32 + lane) * E + i % E; });
  }
  tc::cp_async_wait<0>();
  const int tail = from + vecs * E;
  if (share == 0 && tail < hi) one(tail + lane, tail + lane < hi, BACK);
  const float top = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(st.top)));  // (none is negative or NaN)
  const int owner = __ffs(__ballot_sync(0xffffffffu, st.top == top)) - 1;
  const float s = warp_sum(lane == owner ? st.s : st.s + st.top);
  if (s == s) {
    const int first = st.at == FRONT ? lo + lane : st.at == BACK ? tail + lane : from + (st.at + lane) * E;
    const int vectors = st.at < 0 ? 0 : min(U, (vecs - st.at - lane + 31) / 32);
    const int where = __shfl_sync(0xffffffffu, first | vectors << 24, owner);
    return Stat{st.m, s, top, top > 0.f ? where : 0,
                GREEDY ? (int)__reduce_min_sync(0xffffffffu, (unsigned)st.idx) : NOWHERE};
  }
  Stat slow = NOTHING, out;
  const auto careful = [&](int i) { add_careful(slow, logit(element<F32>(row, i), F32), i, c); };
  if (share == 0 && lane < head) careful(lo + lane);
  for (int block = share * BLOCK; block < vecs; block += step)  // (the same part)
    for (int j = block; j < min(block + BLOCK, vecs - lane); j += 32) {
      Vec<F32> z;
      z.set(v[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) add_careful(slow, logit(z.get(i), F32), from + (j + lane) * E + i, c);
    }
  if (share == 0 && tail + lane < hi) careful(tail + lane);
  __syncwarp();
  out.m = warp_top(slow.m);
  const bool leads = slow.m == out.m && out.m > -INFINITY;
  const int places = __popc(__ballot_sync(0xffffffffu, leads));  // (lanes that have the maximum)
  const float others = leads ? slow.s : slow.m == -INFINITY ? 0.f : (slow.s + 1.f) * tc::ex2_approx((slow.m - out.m) * c);
  out.s = warp_sum(others) + fmaxf((float)places - 1.f, 0.f);
  out.top = places ? 1.f : 0.f;
  out.idx = (int)__reduce_min_sync(0xffffffffu, leads ? (unsigned)slow.idx : (unsigned)NOWHERE);
  out.where = places ? out.idx : 0;
  return out;
}

// What lane `lane` has of the block that weighs most in a row: the element's index (-1: none).
template <bool F32>
__device__ __forceinline__ int of_block(const Stat& st, int lane) {
  constexpr int E = Vec<F32>::E;
  const int first = st.where & 0xFFFFFF, vectors = st.where >> 24;
  if (vectors == 0) return lane == 0 ? first : -1;
  return lane / E < vectors ? first + lane / E * (32 * E) + lane % E : -1;
}

// What turns an element of a row into its probability.
struct Law {
  const void* row;
  bool f32, probs;
  float m, inv;  // reference and 1 / sum (logits)
};

// log2(e) / temperature in two floats.
struct Rate {
  float hi, lo;
};

// 2^((z - m) rate): the roundings of the argument are carried along (an argument of 2^7 has steps of 2^-17).
__device__ __forceinline__ float weight(float z, float m, const Rate& r) {
  const float d = z - m, y = d * r.hi;
  if (!(y > -150.f)) return 0.f;
  const float e = fmaf(d, r.hi, -y) + d * r.lo;
  return tc::ex2_approx(y) * fmaf(e, LN2F, 1.f);
}
// Whether u q(x) < p(x) for logits z of the target's row and y of the draft's, as u < p(x) / q(x): the quotient stands
// where both probabilities are too small for a float.  Quotients of 2^150 and more or less, and those whose exponents leave fp32 (a
// logit of -1e38 does so at temperature 1), are decided by the difference of the exponents in fp64, which holds any of them.
__device__ __forceinline__ bool keeps(float u, float z, const Stat& p, float y, const Stat& q, const Rate& r) {
  if (z == -INFINITY) return false;
  if (y == -INFINITY) return true;
  const float dp = z - p.m, dq = y - q.m, a = dp * r.hi, b = dq * r.hi;
  const float e = (fmaf(dp, r.hi, -a) + dp * r.lo) - (fmaf(dq, r.hi, -b) + dq * r.lo), d = a - b, sum = d + e;
  if (!(fabsf(sum) < 150.f)) {  // (NaN too)
    const double far = (((double)z - p.m) - ((double)y - q.m)) * r.hi;
    return u < tc::ex2_approx((float)fmin(fmax(far, -1000.0), 1000.0)) * ((q.s + q.top) / (p.s + p.top));
  }
  return u < tc::ex2_approx(sum) * fmaf((d - sum) + e, LN2F, 1.f) * ((q.s + q.top) / (p.s + p.top));
}

__device__ __forceinline__ Law law_from(const void* row, bool f32, bool probs, const Stat& st) {
  const float sum = st.s + st.top;
  return Law{row, f32, probs, st.m, sum > 0.f ? 1.f / sum : 0.f};
}

__device__ __forceinline__ float law_of(const Law& l, float x, const Rate& r) {
  if (l.probs) return prob(x);
  return l.m == -INFINITY ? 0.f : weight(logit(x, l.f32), l.m, r) * l.inv;
}

// log p of element i, x, by a warp: over a half from the sum of the other weights, for which each lane has an element y, of index
// j, of the row's heaviest block (error against float64 5e-7 of log p at worst; 7e-4 where p is 0.9995 from a sum with p in it:
// 2 x 4 rows of 32000 0.6 us, 256 x 5 rows of 131072 2 of 133, greedy ones 5 of 71); else of the probability itself, whose error stays that of a weight (a difference of two
// logarithms has the error of the larger); where it is too small for that, of its parts.
__device__ __noinline__ float log_of(bool f32, bool probs, Stat st, float x, int i, float y, int j, Rate r, float temp) {
  const Law l = law_from(nullptr, f32, probs, st);
  const float p = law_of(l, x, r);
  if (!l.probs && p > 0.5f && __any_sync(0xffffffffu, j == i)) {
    const float rest = st.s + warp_sum(j < 0 || j == i ? 0.f : weight(y, st.m, r));
    return -log1pf(rest / weight(logit(x, l.f32), st.m, r));
  }
  return l.probs || p > 1e-30f ? logf(p) : (logit(x, l.f32) - l.m) / temp + logf(l.inv);
}

struct Best {
  float key;
  int idx;
  float x;  // the target's element there
};
__device__ __forceinline__ void take(Best& a, const Best& b) {
  if (b.key > a.key || (b.key == a.key && b.idx < a.idx)) a = b;
}

// The race over elements [lo, hi): r(x) / noise(x), r = p, p without `skip`, or (minus) max(p - q, 0).  Of most elements
// only a quick upper bound of p is computed: it has to pass the best key of the CTA so far, and the draft's row is
// read for those that do.  `top` (shared, 0 at first) holds that key's bits.
template <int NT, int RING, bool F32>
__device__ __forceinline__ Best race(const Law& p, const Law& q, bool minus, int skip, const float* noise, int lo, int hi,
                                     const Rate& r, uint4* ring, int* top) {
  // A warp takes chunks of 8 elements, H of them a lane, as many vectors as four groups and more of them leave room for.
  constexpr int H = F32 ? 1 : 2, E = 8 * H, STEP = 32 * E, SIZE = F32 ? 4 : 2, GROUP = STEP * (SIZE + 4);
  constexpr int GROUPS = RING / GROUP, STRIDE = NT / 32 * STEP;
  Best best = {0.f, NOWHERE, 0.f};
  if (!p.probs && p.m == -INFINITY) return best;
  // An element's quick weight is x itself, or 2^((x - m) c); times scale it is its probability but for 2^-11 of it.
  const float c = r.hi, unit = (1.f - 0x1p-10f) / (p.probs ? 1.f : p.inv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  const auto enter = [&](int i, float x, float e) {
    float w = law_of(p, x, r);
    if (minus) w -= law_of(q, element(q.row, i, q.f32), r);
    const float key = i == skip ? 0.f : __fdividef(w, e);
    if (key > best.key || (key == best.key && key > 0.f && i < best.idx)) best = Best{key, i, x};
  };

  // the part whose vectors are whole, in chunks of 8 elements
  const uintptr_t begin = reinterpret_cast<uintptr_t>(at(p.row, lo, F32));
  const int from = min(hi, lo + (int)((16 - (begin & 15)) & 15) / SIZE), count = (hi - from) / 8 * 8;
  const uint8_t* prow = reinterpret_cast<const uint8_t*>(at(p.row, from, F32)) + lane * 16;
  const float* nrow = noise + from;
  const bool whole = (reinterpret_cast<uintptr_t>(nrow) & 15) == 0;
  uint8_t* mine = reinterpret_cast<uint8_t*>(ring) + warp * RING;
  // (elements as they lie in memory: the target's, then the noise's, which is copied word by word where its row begins
  // off the target's boundaries)
  const auto fetch = [&](int i, int group) {
    uint8_t* to = mine + group * GROUP;
    const int n = min(STEP, count - i);
    if (n > 0) {
#pragma unroll
      for (int u = 0; u < STEP * SIZE / 512; ++u)
        if ((u * 32 + lane) * (16 / SIZE) < n) tc::cp_async16(to + u * 512 + lane * 16, prow + (int64_t)i * SIZE + u * 512, 16);
      to += STEP * SIZE;
      if (whole) {
#pragma unroll
        for (int u = 0; u < STEP / 128; ++u)
          if (u * 128 + lane * 4 < n) tc::cp_async16(to + u * 512 + lane * 16, nrow + i + u * 128 + lane * 4, 16);
      } else {
#pragma unroll
        for (int u = 0; u < STEP / 32; ++u)
          if (u * 32 + lane < n) tc::cp_async4(to + u * 128 + lane * 4, nrow + i + u * 32 + lane);
      }
    }
    tc::cp_async_commit();
  };
  const uint64_t c2 = pack(c, c), m2 = pack(-p.m, -p.m);
  int to = 0, use = 0;
  for (int i0 = warp * STEP - (GROUPS - 1) * STRIDE; i0 < count; i0 += STRIDE) {
    __syncwarp();  // (the group that is filled now has been read by every lane)
    fetch(i0 + (GROUPS - 1) * STRIDE, to);
    to = to == GROUPS - 1 ? 0 : to + 1;
    if (i0 < 0) continue;  // (the first groups)
    tc::cp_async_wait<GROUPS - 1>();
    __syncwarp();
    const uint8_t* group = mine + use * GROUP;
    use = use == GROUPS - 1 ? 0 : use + 1;
    // (chunk h of the lane: elements i0 + 256 h + 8 lane on, there if h * 256 < n)
    const uint8_t* gx = group + lane * 8 * SIZE;
    const float* ge = reinterpret_cast<const float*>(group + STEP * SIZE) + lane * 8;
    const int n = count - i0 - lane * 8;
    uint32_t done = 0;  // candidates that have been looked at
    while (true) {
      const float bar = __int_as_float(*(volatile int*)top) * unit;
      const uint64_t bar2 = pack(-bar, -bar);
      uint64_t over[E / 2];
      float most = 0.f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        Vec<F32> x[SIZE / 2];
#pragma unroll
        for (int v = 0; v < SIZE / 2; ++v) x[v].set(*reinterpret_cast<const uint4*>(gx + h * 256 * SIZE + v * 16));
        const float4 e0 = *reinterpret_cast<const float4*>(ge + h * 256), e1 = *reinterpret_cast<const float4*>(ge + h * 256 + 4);
        const uint64_t e[4] = {pack(e0.x, e0.y), pack(e0.z, e0.w), pack(e1.x, e1.y), pack(e1.z, e1.w)};
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          constexpr int PER = 16 / SIZE;
          uint64_t w = pack(x[k / PER].get(k % PER), x[k / PER].get(k % PER + 1));
          if (!p.probs) {
            const uint64_t y = mul2(add2(w, m2), c2);
            w = pack(tc::ex2_approx(low(y)), tc::ex2_approx(high(y)));
          }
          w = fma2(e[k / 2], bar2, w);
          over[h * 4 + k / 2] = w;
          if (h * 256 < n) most = fmaxf(most, fmaxf(low(w), high(w)));
        }
      }
      if (!__any_sync(0xffffffffu, most > 0.f)) break;
      // each lane looks at the candidate that lies farthest over the bar, which may raise it for the others
      int pick = -1;
      most = 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float w = k & 1 ? high(over[k / 2]) : low(over[k / 2]);
        if (w > most && k / 8 * 256 < n && !(done >> k & 1)) most = w, pick = k;
      }
      if (!__any_sync(0xffffffffu, pick >= 0)) break;
      if (pick >= 0) {
        done |= 1u << pick;
        const int k = pick / 8 * 256 + pick % 8;
        enter(from + i0 + lane * 8 + k, element<F32>(gx, k), ge[k]);
      }
      const int t = __reduce_max_sync(0xffffffffu, __float_as_int(best.key));
      if (lane == 0) atomicMax(top, t);
      __syncwarp();
    }
  }
  tc::cp_async_wait<0>();
  __syncwarp();
  // the elements before and behind the chunks, fewer than 8 each
  const int front = from - lo, rest = from + count, edge = front + hi - rest;
  if ((int)threadIdx.x < edge) {
    const int i = (int)threadIdx.x < front ? lo + (int)threadIdx.x : rest + (int)threadIdx.x - front;
    enter(i, element<F32>(p.row, i), noise[i]);
  }
  return best;
}

struct Args {
  dsv4_draft_verify_params p;
  int rows;  // of a group
};

template <int NT, int DEPTH, int CTAS, bool F32>
__global__ void __launch_bounds__(NT, CTAS) verify_kernel(const __grid_constant__ Args a) {
  constexpr int NW = NT / 32;
  static_assert(MAX_ROWS <= NW, "a warp a row of a group");
  const dsv4_draft_verify_params& p = a.p;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / C;
  extern __shared__ uint4 ring[];
  __shared__ Stat part[NW], got[2][2 * MAX_ROWS][MAX_CLUSTER];
  __shared__ Best bpart[NW], bgot[2][MAX_CLUSTER];
  __shared__ Stat fin[2 * MAX_ROWS];
  __shared__ int stands[MAX_ROWS], top_key, brought_part[NW], drafted[MAX_ROWS];
  __shared__ float drafted_x[MAX_ROWS];
  if (tid == 0) top_key = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = p.q_start[b], t1 = p.q_start[b + 1];
  float temp = p.temperature ? p.temperature[b] : 1.f;
  // Draft rows in order: one for every token but the first of each sequence, so the row of token t + 1 is t less the sequences
  // before b that brought any token.  (The loads lie beside those above: 2 x 4 rows 0.3 us, 256 x 5 rows nothing, 8000 x 2 rows of 100
  // logits 261 us for 239 with rows given by name.)
  if (p.draft != nullptr && p.draft_row == nullptr) {
    int brought = 0;
#pragma unroll 8
    for (int j = tid; j < b; j += NT) brought += p.q_start[j + 1] > p.q_start[j];
    brought = __reduce_add_sync(0xffffffffu, brought);
    if (lane == 0) brought_part[warp] = brought;
  }
  if (t0 < 0 || t1 < t0 || t1 > p.T || t1 - t0 > p.max_q_len) {  // (the same for the whole cluster)
    if (rank == 0 && tid == 0) atomicOr(&g_flags_vf, FLAG_PAGE);
    return;
  }
  const int n = t1 - t0;
  int32_t* out = p.out_tokens + (int64_t)b * p.max_q_len;
  float* logp = p.logp ? p.logp + (int64_t)b * p.max_q_len : nullptr;
  if (n == 0) {
    if (rank == 0) {
      for (int i = tid; i < p.max_q_len; i += NT) {
        out[i] = -1;
        if (logp) logp[i] = 0.f;
      }
      if (tid == 0) p.n_out[b] = 0;
    }
    return;
  }
  cluster.sync();  // every CTA's shared memory is there to be written
  int64_t brought = 0;
  if (p.draft != nullptr && p.draft_row == nullptr)
    for (int w = 0; w < NW; ++w) brought += brought_part[w];
  const auto draft_row_of = [&](int64_t t) { return p.draft_row ? (int64_t)p.draft_row[t + 1] : t - brought; };
  const bool greedy = p.noise == nullptr || !(temp > 0.f);
  temp = greedy ? 1.f : fminf(fmaxf(temp, 1e-30f), 1e30f);
  Rate rate;
  rate.hi = LOG2E_HI / temp;
  rate.lo = rate.hi < 1e30f ? (fmaf(-rate.hi, temp, LOG2E_HI) + LOG2E_LO) / temp : 0.f;
  const bool df32 = p.draft_dtype == DSV4_F32;
  const bool drafted_law = p.draft != nullptr && !greedy;
  const int per = ((p.vocab + C - 1) / C + 7) & ~7, lo = min(p.vocab, rank * per), hi = min(p.vocab, lo + per);
  const bool target_task = !p.target_probs || greedy, draft_task = drafted_law && !p.draft_probs;
  const int tasks_a_row = (target_task ? 1 : 0) + (draft_task ? 1 : 0);

  int last = -1, par = 0;  // the row that the sequence's last token comes from
  bool all = false, residual = false;
  Law lp = {}, lq = {};
  const bool logs = rank == 0 && logp != nullptr && target_task;
  int last_warp = 0, j = -1;
  float y = 0.f;
  const auto write = [&](int i, int token, float z) {  // a warp's row's token
    if (lane == 0) out[i] = token;
    if (!logp) return;
    const float l = log_of(F32, p.target_probs != 0, target_task ? fin[warp * tasks_a_row] : Stat{}, z, token, y, j, rate, temp);
    if (lane == 0) logp[i] = l;
  };
  Best best = {0.f, NOWHERE, 0.f};
  for (int i0 = 0; last < 0; i0 += a.rows) {
    const int rows = min(a.rows, n - i0), tasks = rows * tasks_a_row;
    // each row's drafted successor
    int x = -1;
    int64_t qrow = -1;
    float zx = 0.f, yx = 0.f, ux = 0.f;
    if (tid < rows && i0 + tid + 1 < n) {
      const int t = t0 + i0 + tid;
      x = p.tokens[t + 1];
      const bool in = x >= 0 && x < p.vocab;
      if (in) zx = element(p.target, (int64_t)t * p.target_stride + x, F32);
      if (!greedy) ux = p.u[t + 1];
      if (drafted_law) {
        qrow = draft_row_of(t);
        if (qrow < 0 || qrow >= p.draft_rows) qrow = -1;
        if (in && qrow >= 0) yx = element(p.draft, qrow * p.draft_stride + x, df32);
      }
      if (rank == 0 && (!in || (drafted_law && qrow < 0))) atomicOr(&g_flags_vf, FLAG_PAGE);
      if (!in) x = -1;
    }
    if (tasks > 0) {
      // warp w works on task w % tasks (where there are more tasks than warps, on every NW-th)
      for (int k = tasks < NW ? warp % tasks : warp; k < tasks; k += NW) {
        const int share = tasks < NW ? warp / tasks : 0, shares = tasks < NW ? (NW - 1 - k) / tasks + 1 : 1;
        const int i = i0 + k / tasks_a_row;
        const int64_t t = t0 + i;
        const bool is_target = target_task && k % tasks_a_row == 0;
        int64_t d = 0;
        if (!is_target) {
          d = i + 1 < n ? draft_row_of(t) : -1;
          if (d >= p.draft_rows) d = -1;
        }
        const bool f32 = is_target ? F32 : df32;
        const void* row = is_target ? at(p.target, t * p.target_stride, F32) : at(p.draft, d * p.draft_stride, df32);
        Stat st = NOTHING;
        if (d >= 0) {
          if (greedy)
            st = f32 ? scan_row<NT, DEPTH, true, true>(row, lo, hi, share, shares, rate.hi, ring)
                     : scan_row<NT, DEPTH, false, true>(row, lo, hi, share, shares, rate.hi, ring);
          else
            st = f32 ? scan_row<NT, DEPTH, true, false>(row, lo, hi, share, shares, rate.hi, ring)
                     : scan_row<NT, DEPTH, false, false>(row, lo, hi, share, shares, rate.hi, ring);
        }
        if (tasks < NW) {
          if (lane == 0) part[warp] = st;
        } else if (lane < C) {
          *cluster.map_shared_rank(&got[par][k][rank], lane) = st;
        }
      }
      if (tasks < NW) {
        __syncthreads();
        if (tid < tasks) {
          Stat sum = part[tid];
          for (int w = tid + tasks; w < NW; w += tasks) merge(sum, part[w], rate.hi);
          for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&got[par][tid][rank], r) = sum;
        }
      }
      cluster.sync();
      if (tid < tasks) {
        Stat sum = got[par][tid][0];
        for (int r = 1; r < C; ++r) merge(sum, got[par][tid][r], rate.hi);
        fin[tid] = sum;
      }
      __syncthreads();
      par ^= 1;
    }
    // warp w has row w's heaviest block brought, for the logarithm of the row's token
    y = -INFINITY, j = -1;
    if (logs && warp < rows) {
      j = of_block<F32>(fin[warp * tasks_a_row], lane);
      if (j >= 0) y = logit(element<F32>(at(p.target, (t0 + i0 + warp) * p.target_stride, F32), j), F32);
    }
    if (tid < rows) {
      const Stat ts = target_task ? fin[tid * tasks_a_row] : Stat{};
      const Stat ds = draft_task ? fin[tid * tasks_a_row + tasks_a_row - 1] : Stat{};
      bool ok = false;
      if (x >= 0) {
        if (greedy) {
          ok = ts.m > (p.target_probs ? 0.f : -INFINITY) && x == ts.idx;
        } else if (draft_task && !p.target_probs) {
          ok = qrow >= 0 && keeps(ux, logit(zx, F32), ts, logit(yx, df32), ds, rate);
        } else {
          const Law law = law_from(nullptr, F32, p.target_probs != 0, ts);
          const float px = law_of(law, zx, rate);
          if (!drafted_law) {
            ok = ux < px || (ux == 0.f && !p.target_probs && logit(zx, F32) > -INFINITY);
          } else if (qrow >= 0) {
            const Law dlaw = law_from(nullptr, df32, p.draft_probs != 0, ds);
            ok = ux * law_of(dlaw, yx, rate) < px;
          }
        }
      }
      stands[tid] = ok;
      drafted[tid] = x, drafted_x[tid] = zx;
    }
    __syncthreads();
    int stay = 0;
    while (stay < rows && stands[stay]) ++stay;
    if (stay < rows) {
      last = i0 + stay;
      const int64_t t = t0 + last;
      all = last == n - 1;
      const Stat ts = target_task ? fin[stay * tasks_a_row] : Stat{};
      if (greedy && ts.m > (p.target_probs ? 0.f : -INFINITY)) best = Best{0.f, ts.idx, ts.m};
      lp = law_from(at(p.target, t * p.target_stride, F32), F32, p.target_probs != 0, ts);
      last_warp = stay;
      if (drafted_law && !all) {
        const int64_t d = draft_row_of(t);
        if (d >= 0 && d < p.draft_rows) {
          const Stat ds = draft_task ? fin[stay * tasks_a_row + tasks_a_row - 1] : Stat{};
          lq = law_from(at(p.draft, d * p.draft_stride, df32), df32, p.draft_probs != 0, ds);
          residual = true;
        }
      }
    }
    if (last < 0 && rank == 0 && warp < rows) write(i0 + warp, drafted[warp], drafted_x[warp]);
    __syncthreads();  // fin and stands are free again
  }

  if (!greedy) {
    const float* noise = p.noise + (int64_t)b * p.noise_stride;
    const int skip = !all && p.draft == nullptr ? p.tokens[t0 + last + 1] : -1;
    for (int round = residual || skip >= 0 ? 0 : 1; round < 2; ++round) {
      const bool minus = residual && round == 0;
      const int not_this = round == 0 ? skip : -1;
      Best mine = race<NT, U * DEPTH * 512, F32>(lp, lq, minus, not_this, noise, lo, hi, rate, ring, &top_key);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Best y = {__shfl_xor_sync(0xffffffffu, mine.key, o), __shfl_xor_sync(0xffffffffu, mine.idx, o),
                        __shfl_xor_sync(0xffffffffu, mine.x, o)};
        take(mine, y);
      }
      if (lane == 0) bpart[warp] = mine;
      __syncthreads();
      if (tid < C) {
        mine = bpart[0];
        for (int w = 1; w < NW; ++w) take(mine, bpart[w]);
        *cluster.map_shared_rank(&bgot[round][rank], tid) = mine;
      }
      cluster.sync();
      best = bgot[round][0];
      for (int r = 1; r < C; ++r) take(best, bgot[round][r]);
      if (best.key > 0.f) break;
    }
  }
  if (rank != 0) return;
  const bool found = best.idx != NOWHERE;
  const bool kept = warp < last_warp;  // (of the last group, whose rows the warps still have)
  if (kept || (warp == last_warp && found))
    write(last - last_warp + warp, kept ? drafted[warp] : best.idx, kept ? drafted_x[warp] : best.x);
  for (int i = last + found + tid; i < p.max_q_len; i += NT) {
    out[i] = -1;
    if (logp) logp[i] = 0.f;
  }
  if (tid == 0) p.n_out[b] = last + (found ? 1 : 0);
}

template <int NT, int DEPTH, int CTAS, bool F32>
cudaError_t launch(const Args& a, int cluster, cudaStream_t s) {
  constexpr int RING = NT * U * DEPTH * 16;
  const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(verify_kernel<NT, DEPTH, CTAS, F32>), RING);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.p.B * cluster);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = RING;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, verify_kernel<NT, DEPTH, CTAS, F32>, a));
}

}  // namespace loop

cudaError_t launch_draft_verify(const dsv4_draft_verify_params& p, cudaStream_t s) {
  if (p.B == 0) return cudaSuccess;
  // As many CTAs a sequence as the SMs can hold at once, two each (2 sequences of 32000 logits: 8 CTAs 11.7 us, 4 14.0, 1 28;
  // 64 of 131072 with probabilities of the draft: 4 CTAs 36.3 us, 2 41.7, 8 45.4; 200 x 4 rows of 131072: 1 CTA 103 us, 2 113, but 200
  // x up to 3 rows of 100003, half of them greedy, 45 and 40),
  // of 4000 logits a row at least (22 sequences of 4000: 1 CTA 10.1 us, 2 11.7, 8 14.5; of 16000: 4 CTAs 12.4, 8 13.1, 1 17.5).
  int cluster = 1;
  while (cluster < loop::MAX_CLUSTER && (int64_t)p.B * cluster * 2 <= 2 * num_sms() && p.vocab >= 8000 * cluster) cluster *= 2;
  // Rows in one group share the exchange between the CTAs and their waits (400 sequences of 8000 logits, four rows each:
  // 8 rows a group 31.8 us, 1 52.5), but all of them are read (256 of 131072, five rows each: 8 rows a group 159 us, 1 133):
  // rows of 131072 logits a CTA in all.
  const int slice = (p.vocab + cluster - 1) / cluster, rows = 131072 / slice;
  const loop::Args a = {p, rows < 1 ? 1 : rows > loop::MAX_ROWS ? loop::MAX_ROWS : rows};
  return p.target_dtype == DSV4_F32 ? loop::launch<256, 6, 2, true>(a, cluster, s) : loop::launch<256, 6, 2, false>(a, cluster, s);
}

cudaError_t read_flags_loop_verify(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_vf, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_vf, &z, sizeof(z));
}

}  // namespace dsv4
