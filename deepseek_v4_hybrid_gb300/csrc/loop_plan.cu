// Batch plan: pages given back and taken, block tables, q_start and kv_len, positions and slots of a step.
//
// Everything follows from prefix sums over the requests: tokens, pages given back and pages taken.  A CTA holds the
// sums of all requests in shared memory; then pages and tokens are flat lists whose items find their request by
// a binary search.
#include "loop_common.cuh"
#include "tmap.h"

namespace dsv4 {

static __device__ unsigned int g_flags_pl = 0;

namespace loop {

constexpr int MAX_CTX = 1 << 30;

struct Request {
  int c, n;  // rows kept, tokens wanted
  bool ok;
};

// Pages of a request in one cache.  Table entries [first, held) are its own; [first, lo) and [hi, held) are given
// back, `take` entries from `held` on are wanted.
struct Pages {
  int first, held, lo, hi, take;
};

__device__ __forceinline__ Pages pages_of(const dsv4_plan_cache& k, int b, const Request& r, bool& ok) {
  Pages g;
  g.held = k.held[b];
  g.first = k.window > 0 ? k.first[b] : 0;
  g.lo = g.first, g.hi = g.held, g.take = 0;
  ok = g.first >= 0 && g.held >= g.first && g.held <= k.max_pages_per_seq;
  if (!ok) return g;
  const int rows = r.c + r.n, entries = rows / k.ratio;
  const int need = (int)(((int64_t)entries + k.page_size - 1) / k.page_size);
  if (need > k.max_pages_per_seq) ok = false;
  int seen = 0;  // first page that a token from position c on sees
  if (k.window > 0) {
    seen = max(0, r.c - k.window + 1) / k.page_size;
    if (rows > 0 && seen < g.first) ok = false;
  }
  if (!ok) return g;
  if (rows == 0) {
    g.hi = g.first;  // ended
    return g;
  }
  g.lo = min(g.held, max(g.first, seen));
  g.hi = min(g.held, max(need, g.lo));
  g.take = max(0, need - g.held);
  return g;
}

__device__ __forceinline__ Request request_of(const dsv4_batch_plan_params& p, int b) {
  Request r;
  const int64_t c = (int64_t)p.ctx[b] + (p.ctx_add ? p.ctx_add[b] : 0);
  r.n = p.n_new[b];
  r.ok = c >= 0 && r.n >= 0 && c + r.n <= MAX_CTX;
  r.c = r.ok ? (int)c : 0;
  if (!r.ok) return r;
  for (int g = 0; g < p.num_caches && r.ok; ++g) pages_of(p.caches[g], b, r, r.ok);
  return r;
}

// Exclusive sums of NV values over the block's threads; tot[v] (shared) gets the whole sums.
template <int NV>
__device__ __forceinline__ void block_scan(uint32_t (&v)[NV], uint32_t (*warp_sums)[32], uint32_t* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t own[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) own[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += y;
    }
  }
  __syncthreads();  // (a scan before this one has read the sums)
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < NV; ++i) warp_sums[i][warp] = v[i];
  __syncthreads();
  for (int i = warp; i < NV; i += warps) {
    uint32_t x = lane < warps ? warp_sums[i][lane] : 0;
    const uint32_t mine = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane < warps) warp_sums[i][lane] = x - mine;
    if (lane == 31) tot[i] = x;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] += warp_sums[i][warp] - own[i];
}

// The request that item j of a list with these starts belongs to: the last b < B with start[b] <= j.
__device__ __forceinline__ int owner(const uint32_t* start, int B, uint32_t j) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= j)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int G>
__global__ void __launch_bounds__(1024) plan_kernel(const __grid_constant__ dsv4_batch_plan_params p) {
  extern __shared__ uint32_t sums[];
  __shared__ uint32_t warp_sums[1 + 2 * G][32], total[1 + 2 * G], run_total[1 + G];
  const int B = p.B, tid = threadIdx.x, nt = blockDim.x;
  uint32_t* token0 = sums;                 // [B + 1] first token of each request
  int* kept = (int*)(token0 + B + 1);      // [B + 1] rows kept
  uint32_t* take0 = (uint32_t*)kept + B + 1;   // [G][B + 1] first page taken
  uint32_t* give0 = take0 + G * (B + 1);   // [G][B + 1] first page given back
  pdl_wait();
  pdl_launch_dependents();
  const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const uint32_t T = (uint32_t)p.T;

  // what every request wants (a count over T is as good as T + 1: sums stay below 2^32)
  uint32_t v[1 + 2 * G] = {};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    kept[b] = r.ok ? r.c : -1;
    if (!r.ok) {
      bad = true;
      continue;
    }
    v[0] += min((uint32_t)r.n, T + 1);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      bool ok;
      const Pages k = pages_of(p.caches[g], b, r, ok);
      v[1 + g] += k.take;
      v[1 + G + g] += (k.lo - k.first) + (k.held - k.hi);
    }
  }
  block_scan<1 + 2 * G>(v, warp_sums, total);
  uint32_t count[G], level[G];  // of the stack: before, and with what was given back
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t n = p.caches[g].num_pages, have = *p.caches[g].free_count;
    count[g] = (uint32_t)max((int64_t)0, min(n, have));
    level[g] = (uint32_t)min(n, (int64_t)count[g] + total[1 + G + g]);
    bad |= have < 0 || have > n || (int64_t)count[g] + total[1 + G + g] > n;
  }
  // who runs
  uint32_t run[1 + G] = {};
  {
    uint32_t at[1 + 2 * G];
#pragma unroll
    for (int i = 0; i < 1 + 2 * G; ++i) at[i] = v[i];
    for (int b = b0; b < b1; ++b) {
      if (kept[b] < 0) {
        token0[b] = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) take0[g * (B + 1) + b] = 0, give0[g * (B + 1) + b] = at[1 + G + g];
        continue;
      }
      const Request r = request_of(p, b);
      const uint32_t n = min((uint32_t)r.n, T + 1);
      at[0] += n;
      bool runs = n == 0 || at[0] <= T;
      uint32_t take[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        bool ok;
        const Pages k = pages_of(p.caches[g], b, r, ok);
        give0[g * (B + 1) + b] = at[1 + G + g];
        take[g] = k.take;
        at[1 + g] += k.take;
        at[1 + G + g] += (k.lo - k.first) + (k.held - k.hi);
        runs = runs && (k.take == 0 || at[1 + g] <= level[g]);
      }
      token0[b] = runs ? n : 0;  // (counts here; turned into sums below)
      run[0] += runs ? n : 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        take0[g * (B + 1) + b] = runs ? take[g] : 0;
        run[1 + g] += runs ? take[g] : 0;
      }
    }
  }
  block_scan<1 + G>(run, warp_sums, run_total);
  for (int b = b0; b < b1; ++b) {
    uint32_t x = token0[b];
    token0[b] = run[0];
    run[0] += x;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      x = take0[g * (B + 1) + b];
      take0[g * (B + 1) + b] = run[1 + g];
      run[1 + g] += x;
    }
  }
  if (tid == 0) {
    token0[B] = run_total[0];
#pragma unroll
    for (int g = 0; g < G; ++g) take0[g * (B + 1) + B] = run_total[1 + g], give0[g * (B + 1) + B] = total[1 + G + g];
  }
  __syncthreads();

  // given back
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const dsv4_plan_cache& k = p.caches[g];
    const uint32_t* start = give0 + g * (B + 1);
    for (uint32_t j = tid; j < total[1 + G + g]; j += nt) {
      const int b = owner(start, B, j);
      const Request r = request_of(p, b);
      bool ok;
      const Pages e = pages_of(k, b, r, ok);
      const int i = (int)(j - start[b]), front = e.lo - e.first;
      const int entry = i < front ? e.first + i : e.hi + i - front;
      if (count[g] + (uint64_t)j < (uint64_t)k.num_pages)
        k.free_pages[count[g] + j] = k.block_table[(int64_t)b * k.max_pages_per_seq + entry];
    }
  }
  __syncthreads();
  // taken
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const dsv4_plan_cache& k = p.caches[g];
    const uint32_t* start = take0 + g * (B + 1);
    for (uint32_t j = tid; j < run_total[1 + g]; j += nt) {
      const int b = owner(start, B, j);
      const int page = k.free_pages[level[g] - 1 - j];
      k.block_table[(int64_t)b * k.max_pages_per_seq + k.held[b] + (j - start[b])] = page;
      bad |= page < 0 || page >= k.num_pages;
    }
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&g_flags_pl, FLAG_PAGE);

  // the batch's state
  for (int b = tid; b < B; b += nt) {
    const Request r = request_of(p, b);
    const int n = (int)(token0[b + 1] - token0[b]);
    p.kv_len[b] = r.ok ? r.c + n : 0;
    p.q_start[b] = (int)token0[b];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const dsv4_plan_cache& k = p.caches[g];
      int first = k.window > 0 ? k.first[b] : 0, held = k.held[b];
      if (r.ok) {
        bool ok;
        const Pages e = pages_of(k, b, r, ok);
        const bool over = r.c + r.n == 0;
        first = over ? 0 : e.lo;
        held = over ? 0 : e.hi + (int)(take0[g * (B + 1) + b + 1] - take0[g * (B + 1) + b]);
      }
      k.held_out[b] = held;
      if (k.window > 0) k.first_out[b] = first;
    }
    if (p.ctx_out) p.ctx_out[b] = r.ok ? r.c : p.ctx[b];
  }
  if (tid == 0) {
    p.q_start[B] = (int)token0[B];
#pragma unroll
    for (int g = 0; g < G; ++g) *p.caches[g].free_count_out = (int)(level[g] - run_total[1 + g]);
  }
  // positions and slots
  for (uint32_t t = tid; t < T; t += nt) {
    const bool real = t < token0[B];
    const int b = real ? owner(token0, B, t) : 0;
    const int pos = real ? kept[b] + (int)(t - token0[b]) : -1;
    if (p.positions) p.positions[t] = pos;
    if (p.token_seq) p.token_seq[t] = real ? b : -1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const dsv4_plan_cache& k = p.caches[g];
      if (!k.slots) continue;
      int64_t slot = -1;
      if (real && (pos + 1) % k.ratio == 0) {
        const int entry = pos / k.ratio;
        const int page = __ldcg(k.block_table + (int64_t)b * k.max_pages_per_seq + entry / k.page_size);
        if (page >= 0 && page < k.num_pages) slot = (int64_t)page * k.page_size + entry % k.page_size;
      }
      k.slots[t] = slot;
    }
  }
}

}  // namespace loop

namespace {
template <int G>
cudaError_t launch_plan(const dsv4_batch_plan_params& p, cudaStream_t s) {
  const size_t smem = (size_t)(2 + 2 * G) * (p.B + 1) * 4;
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(loop::plan_kernel<G>),
                                          (2 + 2 * G) * (DSV4_PLAN_MAX_REQUESTS + 1) * 4);
  if (e != cudaSuccess) return e;
  return launch_pdl(loop::plan_kernel<G>, dim3(1), dim3(1024), smem, s, true, p);
}
}  // namespace

cudaError_t launch_batch_plan(const dsv4_batch_plan_params& p, cudaStream_t s) {
  switch (p.num_caches) {
    case 1: return launch_plan<1>(p, s);
    case 2: return launch_plan<2>(p, s);
    case 3: return launch_plan<3>(p, s);
    default: return launch_plan<4>(p, s);
  }
}

cudaError_t read_flags_loop_plan(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_pl, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_pl, &z, sizeof(z));
}

}  // namespace dsv4
