// Verification of drafted tokens.
//
// A cluster of CTAs takes a sequence, each CTA the same slice of the vocabulary of every row.  Rows are taken in groups:
// the warps go over the slices of a group's rows once, with the running maximum and the sum of e^(z - max) of a
// softmax (in 32-bit floats), the CTAs exchange these through distributed shared memory, and every CTA
// finds by itself how far the drafted tokens stand.  The row where they end is read once more, from the L2 cache,
// for the race argmax r(x) / noise(x), whose winners are exchanged the same way.  Rows behind that one are not read.
#include <cooperative_groups.h>

#include "loop_common.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace dsv4 {

static __device__ unsigned int g_flags_vf = 0;

namespace loop {

namespace cg = cooperative_groups;

constexpr int NT = 512, NW = NT / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_ROWS = NW / 2;  // rows of a group: a warp at least for each row of target and draft
constexpr float LOG2E_HI = 1.44269502162933349609375f, LOG2E_LO = 1.92596299112661746887e-8f, LN2F = 0.69314718055994531f;
constexpr float MAX_F32 = 3.4028234663852886e38f;

// Maximum, its first index, and the sum of 2^((z - m) c) of a part of a row.
struct Stat {
  float m, s;
  int idx;
};

__device__ __forceinline__ void merge(Stat& a, const Stat& b, float c) {
  if (b.m == -INFINITY) return;
  if (b.m > a.m) {
    a.s = b.s + (a.m == -INFINITY ? 0.f : a.s * tc::ex2_approx((a.m - b.m) * c));
    a.m = b.m, a.idx = b.idx;
  } else {
    a.s += b.s * tc::ex2_approx((b.m - a.m) * c);
    if (b.m == a.m) a.idx = min(a.idx, b.idx);
  }
}

// A logit as it counts: NaN as -inf, +inf as the largest value.
__device__ __forceinline__ float logit(float x) { return fminf(fmaxf(x, -INFINITY), MAX_F32); }
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

// Adds N logits with indices index(0) < index(1) < ... to st.
template <int N, typename I>
__device__ __forceinline__ void add(Stat& st, const float (&z)[N], float c, I index) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, z[i]);
  if (top > st.m) {
    st.s = st.m == -INFINITY ? 0.f : st.s * tc::ex2_approx((st.m - top) * c);
    st.m = top;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (z[i] == top) st.idx = index(i);
  }
  if (st.m == -INFINITY) return;
#pragma unroll
  for (int i = 0; i < N; ++i) st.s += tc::ex2_approx((z[i] - st.m) * c);
}

// Elements [lo, hi) of a row of logits, by lane `lane` of `lanes` threads.
template <bool F32>
__device__ __forceinline__ Stat scan_row(const void* row, int lo, int hi, int lane, int lanes, float c) {
  constexpr int E = F32 ? 4 : 8, U = F32 ? 4 : 2;  // elements of 16 bytes, loads in flight
  Stat st = {-INFINITY, 0.f, 0x7FFFFFFF};
  const uintptr_t a = reinterpret_cast<uintptr_t>(at(row, lo, F32));
  const int head = min(hi - lo, (int)((16 - (a & 15)) & 15) / (F32 ? 4 : 2));  // elements before the first whole 16 bytes
  if (lane < head) {
    const float z[1] = {logit(element<F32>(row, lo + lane))};
    add<1>(st, z, c, [&](int) { return lo + lane; });
  }
  const int from = lo + head, vecs = (hi - from) / E;
  const uint4* v = reinterpret_cast<const uint4*>(at(row, from, F32));
  for (int j = lane; j < vecs; j += U * lanes) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t none = F32 ? 0xFF800000u : 0xFF80FF80u;
      raw[u] = make_uint4(none, none, none, none);
      if (j + u * lanes < vecs) raw[u] = v[j + u * lanes];
    }
    float z[U * E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (F32) {
          z[u * E + i] = logit(__uint_as_float(w[i]));
        } else {
          z[u * E + 2 * i] = logit(__uint_as_float(w[i] << 16));
          z[u * E + (2 * i + 1) % E] = logit(__uint_as_float(w[i] & 0xFFFF0000u));
        }
      }
    }
    add<U * E>(st, z, c, [&](int i) { return from + (j + i / E * lanes) * E + i % E; });
  }
  const int tail = from + vecs * E + lane;
  if (tail < hi) {
    const float z[1] = {logit(element<F32>(row, tail))};
    add<1>(st, z, c, [&](int) { return tail; });
  }
  return st;
}

__device__ __forceinline__ Stat warp_merge(Stat st, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat y;
    y.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    y.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    y.idx = __shfl_xor_sync(0xffffffffu, st.idx, o);
    // (both lanes of a pair merge in the same order, so that they agree)
    Stat lo = (threadIdx.x & o) ? y : st;
    merge(lo, (threadIdx.x & o) ? st : y, c);
    st = lo;
  }
  return st;
}

// What turns an element of a row into its probability.
struct Law {
  const void* row;
  bool f32, probs;
  float m, inv;  // maximum and 1 / sum (logits)
};

// log2(e) / temperature in two floats.
struct Rate {
  float hi, lo;
};

// 2^((z - m) rate): the argument's rounding is carried along, as the special-function unit's input has 24 bits of
// arguments up to 2^7.
__device__ __forceinline__ float weight(float z, float m, const Rate& r) {
  const float d = z - m, y = d * r.hi;
  if (!(y > -150.f)) return 0.f;
  const float e = fmaf(d, r.hi, -y) + d * r.lo;
  return tc::ex2_approx(y) * fmaf(e, LN2F, 1.f);
}
// Whether u q(x) < p(x) for logits z of the target's row and y of the draft's, as u < p(x) / q(x): the quotient stands
// where both probabilities are too small for a float.
__device__ __forceinline__ bool keeps(float u, float z, const Stat& p, float y, const Stat& q, const Rate& r) {
  if (z == -INFINITY) return false;
  if (y == -INFINITY) return true;
  const float dp = z - p.m, dq = y - q.m, a = dp * r.hi, b = dq * r.hi;
  const float e = (fmaf(dp, r.hi, -a) + dp * r.lo) - (fmaf(dq, r.hi, -b) + dq * r.lo), d = a - b, sum = d + e;
  return u < tc::ex2_approx(sum) * fmaf((d - sum) + e, LN2F, 1.f) * (q.s / p.s);
}

__device__ __forceinline__ float law_of(const Law& l, float x, const Rate& r) {
  if (l.probs) return prob(x);
  return l.m == -INFINITY ? 0.f : weight(logit(x), l.m, r) * l.inv;
}

struct Best {
  float key;
  int idx;
  float x;  // the target's element there
};
__device__ __forceinline__ void take(Best& a, const Best& b) {
  if (b.key > a.key || (b.key == a.key && b.idx < a.idx)) a = b;
}

// The race over elements [lo, hi): r(x) / noise(x), r = p, max(p - q, 0) or p without `skip`.
__device__ __forceinline__ Best race(const Law& p, const Law& q, bool minus, int skip, const float* noise, int lo, int hi,
                                     const Rate& r) {
  Best best = {0.f, 0x7FFFFFFF, 0.f};
  for (int i = lo + (int)threadIdx.x; i < hi; i += NT) {
    const float x = element(p.row, i, p.f32);
    float w = law_of(p, x, r);
    if (minus) w -= law_of(q, element(q.row, i, q.f32), r);
    if (i == skip) w = 0.f;
    const float key = __fdividef(w, noise[i]);
    if (key > best.key) best = Best{key, i, x};
  }
  return best;
}

struct Args {
  dsv4_draft_verify_params p;
  int rows;  // of a group
};

__global__ void __launch_bounds__(NT) verify_kernel(const __grid_constant__ Args a) {
  const dsv4_draft_verify_params& p = a.p;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / C;
  __shared__ Stat part[NW], got[2][2 * MAX_ROWS][MAX_CLUSTER];
  __shared__ Best bpart[NW], bgot[2][MAX_CLUSTER];
  __shared__ Stat fin[2 * MAX_ROWS];
  __shared__ int stands[MAX_ROWS];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = p.q_start[b], t1 = p.q_start[b + 1];
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
  float temp = p.temperature ? p.temperature[b] : 1.f;
  const bool greedy = p.noise == nullptr || !(temp > 0.f);
  temp = greedy ? 1.f : fminf(fmaxf(temp, 1e-30f), 1e30f);
  Rate rate;
  rate.hi = LOG2E_HI / temp;
  rate.lo = rate.hi < 1e30f ? (fmaf(-rate.hi, temp, LOG2E_HI) + LOG2E_LO) / temp : 0.f;
  const bool tf32 = p.target_dtype == DSV4_F32, df32 = p.draft_dtype == DSV4_F32;
  const bool drafted_law = p.draft != nullptr && !greedy;
  const int per = ((p.vocab + C - 1) / C + 7) & ~7, lo = min(p.vocab, rank * per), hi = min(p.vocab, lo + per);
  const int tasks_a_row = (!p.target_probs || greedy ? 1 : 0) + (drafted_law && !p.draft_probs ? 1 : 0);
  const bool target_task = !p.target_probs || greedy;

  int last = -1, par = 0;  // the row that the sequence's last token comes from
  bool all = false, excluded = false;
  Law lp = {}, lq = {};
  int best_idx = 0;
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
      if (in) zx = element(p.target, (int64_t)t * p.target_stride + x, tf32);
      if (!greedy) ux = p.u[t + 1];
      if (drafted_law) {
        qrow = p.draft_row ? p.draft_row[t + 1] : t - b;
        if (qrow < 0 || qrow >= p.draft_rows) qrow = -1;
        if (in && qrow >= 0) yx = element(p.draft, qrow * p.draft_stride + x, df32);
      }
      if (rank == 0 && (!in || (drafted_law && qrow < 0))) atomicOr(&g_flags_vf, FLAG_PAGE);
      if (!in) x = -1;
    }
    if (tasks > 0) {
      // warp w works on task w % tasks
      const int k = warp % tasks, share = warp / tasks, shares = (NW - 1 - k) / tasks + 1;
      const int i = i0 + k / tasks_a_row;
      const bool is_target = target_task && k % tasks_a_row == 0;
      Stat st = {-INFINITY, 0.f, 0x7FFFFFFF};
      const int64_t t = t0 + i;
      if (is_target) {
        const void* row = at(p.target, t * p.target_stride, tf32);
        st = tf32 ? scan_row<true>(row, lo, hi, share * 32 + lane, shares * 32, rate.hi)
                  : scan_row<false>(row, lo, hi, share * 32 + lane, shares * 32, rate.hi);
      } else if (i + 1 < n) {
        const int64_t d = p.draft_row ? p.draft_row[t + 1] : t - b;
        if (d >= 0 && d < p.draft_rows) {
          const void* row = at(p.draft, d * p.draft_stride, df32);
          st = df32 ? scan_row<true>(row, lo, hi, share * 32 + lane, shares * 32, rate.hi)
                    : scan_row<false>(row, lo, hi, share * 32 + lane, shares * 32, rate.hi);
        }
      }
      st = warp_merge(st, rate.hi);
      if (lane == 0) part[warp] = st;
      __syncthreads();
      if (tid < tasks) {
        Stat sum = part[tid];
        for (int w = tid + tasks; w < NW; w += tasks) merge(sum, part[w], rate.hi);
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&got[par][tid][rank], r) = sum;
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
    if (tid < rows) {
      const Stat ts = target_task ? fin[tid * tasks_a_row] : Stat{};
      const Stat ds = drafted_law && !p.draft_probs ? fin[tid * tasks_a_row + tasks_a_row - 1] : Stat{};
      bool ok = false;
      float l = 0.f;
      if (x >= 0) {
        const Law law = {nullptr, tf32, p.target_probs != 0, ts.m, ts.s > 0.f ? 1.f / ts.s : 0.f};
        const float px = law_of(law, zx, rate);
        l = p.target_probs ? logf(px) : (logit(zx) - ts.m) / temp - logf(ts.s);
        if (greedy) {
          ok = ts.m > (p.target_probs ? 0.f : -INFINITY) && x == ts.idx;
        } else if (!drafted_law) {
          ok = ux < px || (ux == 0.f && !p.target_probs && logit(zx) > -INFINITY);
        } else if (qrow >= 0) {
          const Law dlaw = {nullptr, df32, p.draft_probs != 0, ds.m, ds.s > 0.f ? 1.f / ds.s : 0.f};
          ok = p.target_probs || p.draft_probs ? ux * law_of(dlaw, yx, rate) < px
                                               : keeps(ux, logit(zx), ts, logit(yx), ds, rate);
        }
        if (ok && rank == 0) {
          // (written whether or not an earlier one falls: what follows the last token is overwritten below)
          out[i0 + tid] = x;
          if (logp) logp[i0 + tid] = l;
        }
      }
      stands[tid] = ok;
    }
    __syncthreads();
    for (int j = 0; j < rows; ++j) {
      if (stands[j]) continue;
      last = i0 + j;
      const int64_t t = t0 + last;
      all = last == n - 1;
      const Stat ts = target_task ? fin[j * tasks_a_row] : Stat{};
      best_idx = ts.m > (p.target_probs ? 0.f : -INFINITY) ? ts.idx : 0x7FFFFFFF;
      lp = Law{at(p.target, t * p.target_stride, tf32), tf32, p.target_probs != 0, ts.m, ts.s > 0.f ? 1.f / ts.s : 0.f};
      if (drafted_law && !all) {
        const int64_t d = p.draft_row ? p.draft_row[t + 1] : t - b;
        if (d >= 0 && d < p.draft_rows) {
          const Stat ds = p.draft_probs ? Stat{} : fin[j * tasks_a_row + tasks_a_row - 1];
          lq = Law{at(p.draft, d * p.draft_stride, df32), df32, p.draft_probs != 0, ds.m, ds.s > 0.f ? 1.f / ds.s : 0.f};
          excluded = true;
        }
      }
      break;
    }
    __syncthreads();  // fin and stands are free again
  }

  Best best = {0.f, best_idx, 0.f};
  if (!greedy) {
    const float* noise = p.noise + (int64_t)b * p.noise_stride;
    const int skip = !all && p.draft == nullptr ? p.tokens[t0 + last + 1] : -1;
    for (int round = excluded || skip >= 0 ? 0 : 1; round < 2; ++round) {
      Best mine = race(lp, lq, excluded && round == 0, round == 0 ? skip : -1, noise, lo, hi, rate);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Best y = {__shfl_xor_sync(0xffffffffu, mine.key, o), __shfl_xor_sync(0xffffffffu, mine.idx, o),
                        __shfl_xor_sync(0xffffffffu, mine.x, o)};
        take(mine, y);
      }
      if (lane == 0) bpart[warp] = mine;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < NW; ++w) take(mine, bpart[w]);
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&bgot[round][rank], r) = mine;
      }
      cluster.sync();
      best = bgot[round][0];
      for (int r = 1; r < C; ++r) take(best, bgot[round][r]);
      if (best.key > 0.f) break;
    }
  }
  if (rank != 0) return;
  const bool found = best.idx != 0x7FFFFFFF;
  for (int i = last + tid; i < p.max_q_len; i += NT) {
    int token = -1;
    float l = 0.f;
    if (i == last && found) {
      token = best.idx;
      const float x = element(lp.row, token, tf32);
      l = p.target_probs ? logf(prob(x)) : (logit(x) - lp.m) / temp - logf(1.f / lp.inv);
    }
    out[i] = token;
    if (logp) logp[i] = l;
  }
  if (tid == 0) p.n_out[b] = last + (found ? 1 : 0);
}

}  // namespace loop

cudaError_t launch_draft_verify(const dsv4_draft_verify_params& p, cudaStream_t s) {
  if (p.B == 0) return cudaSuccess;
  loop::Args a = {p, 1};
  cudaLaunchConfig_t cfg = {};
  const int cluster = 1;
  cfg.gridDim = dim3((unsigned)p.B * cluster);
  cfg.blockDim = dim3(loop::NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, loop::verify_kernel, a));
}

cudaError_t read_flags_loop_verify(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_vf, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_vf, &z, sizeof(z));
}

}  // namespace dsv4
