// Batch plan: pages given back and taken, block tables, q_start and kv_len, positions and slots of a step.
//
// Everything follows from prefix sums over the requests: tokens, pages given back and pages taken.  Every CTA of one
// cluster holds the sums of all requests in shared memory; then pages and tokens are flat lists, shared out over the
// cluster, whose items find their request by a binary search.  Two cluster barriers: pages given back lie on the stack
// before pages are taken from it, and tables are complete before slots are read from them.
// Bound by latency: a launch, the loads of a request's numbers, the sums, page, table and slot in turn.  64 requests with
// four tokens each 5.5 us; 1000 requests in three caches 13.3 us (15.3 with the caches one after the other); 65k prompt
// tokens 11.4 us (1 MB written, by eight SMs).
#include <cooperative_groups.h>

#include "loop_common.cuh"
#include "tmap.h"

namespace dsv4 {

static __device__ unsigned int g_flags_pl = 0;

namespace loop {

namespace cg = cooperative_groups;

constexpr int MAX_CTX = 1 << 30;

// Quotients of numbers below 2^31 by d <= 2^16 as one product: with 2^s >= d, m = ceil(2^(31 + s) / d) is off by less than
// one, so n m / 2^(31 + s) by less than n / 2^(31 + s) < 1 / d.
struct Div {
  uint32_t m, shift;
  static Div by(uint32_t d) {
    Div v = {0, 31};
    while ((1u << (v.shift - 31)) < d) ++v.shift;
    v.m = (uint32_t)(((1ull << v.shift) + d - 1) / d);
    return v;
  }
  __device__ __forceinline__ int quotient(int n) const { return (int)((uint64_t)(uint32_t)n * m >> shift); }
};

struct Args {
  dsv4_batch_plan_params p;
  Div page[DSV4_PLAN_MAX_CACHES], ratio[DSV4_PLAN_MAX_CACHES];
};

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

// What a request wants: rows kept c (-1: it is left alone), tokens n, and of each cache the pages that it gives back before
// its window (front) and in all, and those that it takes.
template <int G>
struct Wants {
  int c, n, front[G], give[G], take[G];
};

template <int G>
__device__ __forceinline__ Wants<G> wants_of(const Args& a, int b) {
  const dsv4_batch_plan_params& p = a.p;
  Wants<G> w = {};
  int held[G], first[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    held[g] = p.caches[g].held[b];
    first[g] = p.caches[g].window > 0 ? p.caches[g].first[b] : 0;
  }
  const int64_t c = (int64_t)p.ctx[b] + (p.ctx_add ? p.ctx_add[b] : 0);
  w.n = p.n_new[b];
  bool ok = c >= 0 && w.n >= 0 && c + w.n <= MAX_CTX;
  const int rows = ok ? (int)c + w.n : 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const dsv4_plan_cache& k = p.caches[g];
    const int need = a.page[g].quotient(a.ratio[g].quotient(rows) + k.page_size - 1);
    int seen = 0;  // first page that a token from row c on sees
    if (k.window > 0 && ok) seen = a.page[g].quotient(max(0, (int)c - k.window + 1));
    ok = ok && first[g] >= 0 && held[g] >= first[g] && held[g] <= k.max_pages_per_seq && need <= k.max_pages_per_seq &&
         !(k.window > 0 && rows > 0 && seen < first[g]);
    if (rows == 0) {  // ended
      w.give[g] = held[g] - first[g];
    } else {
      const int lo = min(held[g], max(first[g], seen)), hi = min(held[g], max(need, lo));
      w.front[g] = lo - first[g];
      w.give[g] = w.front[g] + held[g] - hi;
      w.take[g] = w.n > 0 ? max(0, need - held[g]) : 0;
    }
  }
  w.c = ok ? (int)c : -1;
  if (!ok) {
    w.n = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) w.front[g] = w.give[g] = w.take[g] = 0;
  }
  return w;
}

template <int G>
__global__ void __launch_bounds__(1024) plan_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint32_t sums[];
  __shared__ uint32_t warp_sums[1 + 2 * G][32], total[1 + 2 * G], run_total[1 + G];
  cg::cluster_group cluster = cg::this_cluster();
  const dsv4_batch_plan_params& p = a.p;
  const int B = p.B, S = B + 1, tid = threadIdx.x, nt = blockDim.x;
  const int all_threads = nt * cluster.num_blocks(), me = tid + nt * cluster.block_rank();
  uint32_t* token0 = sums;        // [B + 1] first token of each request
  int* kept = (int*)(sums + S);   // [B + 1] rows kept, -1: left alone
  uint32_t* take0 = sums + 2 * S;  // [G][B + 1] first page taken
  uint32_t* give0 = take0 + G * S;  // [G][B + 1] first page given back
  uint32_t* fronts = give0 + G * S;  // [G][B + 1] pages given back before the window
  pdl_wait();
  pdl_launch_dependents();
  const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const uint32_t T = (uint32_t)p.T;
  int have[G];
#pragma unroll
  for (int g = 0; g < G; ++g) have[g] = *p.caches[g].free_count;

  // what every request wants (a count over T is as good as T + 1: sums stay below 2^32)
  uint32_t v[1 + 2 * G] = {};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Wants<G> w = wants_of<G>(a, b);
    bad |= w.c < 0;
    kept[b] = w.c;
    v[0] += token0[b] = min((uint32_t)w.n, T + 1);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      v[1 + g] += take0[g * S + b] = w.take[g];
      v[1 + G + g] += give0[g * S + b] = w.give[g];
      fronts[g * S + b] = w.front[g];
    }
  }
  block_scan<1 + 2 * G>(v, warp_sums, total);
  uint32_t count[G], level[G];  // of the stack: before, and with what was given back
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t n = p.caches[g].num_pages;
    count[g] = (uint32_t)max((int64_t)0, min(n, (int64_t)have[g]));
    level[g] = (uint32_t)min(n, (int64_t)count[g] + total[1 + G + g]);
    bad |= have[g] < 0 || have[g] > n || (int64_t)count[g] + total[1 + G + g] > n;
  }
  // who runs: the sums up to a request have to fit
  uint32_t run[1 + G], at[1 + G];
#pragma unroll
  for (int i = 0; i <= G; ++i) run[i] = v[i], at[i] = v[i];
  bool fits = total[0] <= T;
#pragma unroll
  for (int g = 0; g < G; ++g) fits = fits && total[1 + g] <= level[g];
  if (!fits) {  // (the same for all threads)
#pragma unroll
    for (int i = 0; i <= G; ++i) run[i] = 0;
    for (int b = b0; b < b1; ++b) {
      const uint32_t n = token0[b];
      at[0] += n;
      bool runs = n == 0 || at[0] <= T;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t k = take0[g * S + b];
        at[1 + g] += k;
        runs = runs && (k == 0 || at[1 + g] <= level[g]);
      }
      if (!runs) {
        token0[b] = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) take0[g * S + b] = 0;
      }
      run[0] += token0[b];
#pragma unroll
      for (int g = 0; g < G; ++g) run[1 + g] += take0[g * S + b];
    }
    block_scan<1 + G>(run, warp_sums, run_total);
  } else if (tid <= G) {
    run_total[tid] = total[tid];
  }
  const auto start = [](uint32_t& count, uint32_t& sum) {  // a count becomes the sum of those before it
    const uint32_t x = count;
    count = sum;
    sum += x;
  };
  for (int b = b0; b < b1; ++b) {
    start(token0[b], run[0]);
#pragma unroll
    for (int g = 0; g < G; ++g) start(take0[g * S + b], run[1 + g]), start(give0[g * S + b], v[1 + G + g]);
  }
  __syncthreads();
  if (tid == 0) {
    token0[B] = run_total[0];
#pragma unroll
    for (int g = 0; g < G; ++g) take0[g * S + B] = run_total[1 + g], give0[g * S + B] = total[1 + G + g];
  }
  __syncthreads();

  // given back (the loads of all caches side by side, here and below)
  uint32_t gives = 0, takes = 0;  // of the longest list
#pragma unroll
  for (int g = 0; g < G; ++g) gives = max(gives, total[1 + G + g]), takes = max(takes, run_total[1 + g]);
  for (uint32_t j = me; j < gives; j += all_threads) {
    int page[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (j >= total[1 + G + g]) continue;
      const dsv4_plan_cache& k = p.caches[g];
      const uint32_t* first_of = give0 + g * S;
      const int b = owner(first_of, B, j), i = (int)(j - first_of[b]), front = (int)fronts[g * S + b];
      const int entry = i < front ? k.first[b] + i : k.held[b] - (int)(first_of[b + 1] - first_of[b]) + i;
      page[g] = k.block_table[(int64_t)b * k.max_pages_per_seq + entry];
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (j < total[1 + G + g] && count[g] + (uint64_t)j < (uint64_t)p.caches[g].num_pages)
        p.caches[g].free_pages[count[g] + j] = page[g];
  }
  if (gives) cluster.sync();
  // taken (what lies on the stack may have been put there by another CTA: read past L1)
  for (uint32_t j = me; j < takes; j += all_threads) {
    int page[G];
    int64_t to[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (j >= run_total[1 + g]) continue;
      const dsv4_plan_cache& k = p.caches[g];
      page[g] = __ldcg(k.free_pages + (level[g] - 1 - j));
      const uint32_t* first_of = take0 + g * S;
      const int b = owner(first_of, B, j);
      to[g] = (int64_t)b * k.max_pages_per_seq + k.held[b] + (j - first_of[b]);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (j >= run_total[1 + g]) continue;
      p.caches[g].block_table[to[g]] = page[g];
      bad |= page[g] < 0 || page[g] >= p.caches[g].num_pages;
    }
  }
  if (bad) atomicOr(&g_flags_pl, FLAG_PAGE);
  cluster.sync();

  // the batch's state (each request's inputs are read by the thread that writes its outputs, which may be the same)
  for (int b = me; b < B; b += all_threads) {
    const int n = (int)(token0[b + 1] - token0[b]), c = kept[b], wanted = p.n_new[b];
    const int ctx = c >= 0 ? c : p.ctx[b];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const dsv4_plan_cache& k = p.caches[g];
      const int front = (int)fronts[g * S + b], back = (int)(give0[g * S + b + 1] - give0[g * S + b]) - front;
      int first = k.window > 0 ? k.first[b] + front : 0;
      int held = k.held[b] - back + (int)(take0[g * S + b + 1] - take0[g * S + b]);
      if (c == 0 && wanted == 0) first = held = 0;
      k.held_out[b] = held;
      if (k.window > 0) k.first_out[b] = first;
    }
    if (p.ctx_out) p.ctx_out[b] = ctx;
    p.kv_len[b] = c >= 0 ? c + n : 0;
    p.q_start[b] = (int)token0[b];
  }
  if (me == 0) {
    p.q_start[B] = (int)token0[B];
#pragma unroll
    for (int g = 0; g < G; ++g) *p.caches[g].free_count_out = (int)(level[g] - run_total[1 + g]);
  }
  // positions and slots, four tokens a thread
  const uint32_t tokens = token0[B];
  for (uint32_t t = 4 * me; t < T; t += 4 * all_threads) {
    int b = t < tokens ? owner(token0, B, t) : 0;
    int pos[4], seq[4], page[G][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool real = t + i < tokens;
      if (real)
        while (token0[b + 1] <= t + i) ++b;
      pos[i] = real ? kept[b] + (int)(t + i - token0[b]) : -1;
      seq[i] = real ? b : -1;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const dsv4_plan_cache& k = p.caches[g];
        const int entry = a.ratio[g].quotient(pos[i] + 1) - 1;  // (of a token that completes it)
        page[g][i] = -1;
        if (k.slots && real && (entry + 1) * k.ratio == pos[i] + 1)
          page[g][i] = __ldcg(k.block_table + (int64_t)b * k.max_pages_per_seq + a.page[g].quotient(entry));
      }
    }
    const bool four = t + 4 <= T;
    if (four) {
      if (p.positions) *reinterpret_cast<int4*>(p.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.token_seq) *reinterpret_cast<int4*>(p.token_seq + t) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    } else {
      for (int i = 0; i < 4 && t + i < T; ++i) {
        if (p.positions) p.positions[t + i] = pos[i];
        if (p.token_seq) p.token_seq[t + i] = seq[i];
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const dsv4_plan_cache& k = p.caches[g];
      if (!k.slots) continue;
      int64_t slot[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int entry = a.ratio[g].quotient(pos[i] + 1) - 1;
        const bool good = page[g][i] >= 0 && page[g][i] < k.num_pages;
        slot[i] = good ? (int64_t)page[g][i] * k.page_size + entry - a.page[g].quotient(entry) * k.page_size : -1;
      }
      if (four) {
        *reinterpret_cast<longlong2*>(k.slots + t) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(k.slots + t + 2) = make_longlong2(slot[2], slot[3]);
      } else {
        for (int i = 0; i < 4 && t + i < T; ++i) k.slots[t + i] = slot[i];
      }
    }
  }
}

}  // namespace loop

namespace {
template <int G>
cudaError_t launch_plan(const loop::Args& a, int cluster, int threads, cudaStream_t s) {
  const auto bytes = [](int B) { return (size_t)(2 + 3 * G) * (B + 1) * 4; };
  const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(loop::plan_kernel<G>),
                                                (int)bytes(DSV4_PLAN_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes(a.p.B);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, loop::plan_kernel<G>, a));
}
}  // namespace

cudaError_t launch_batch_plan(const dsv4_batch_plan_params& p, cudaStream_t s) {
  loop::Args a = {p, {}, {}};
  for (int g = 0; g < p.num_caches; ++g) {
    a.page[g] = loop::Div::by(p.caches[g].page_size);
    a.ratio[g] = loop::Div::by(p.caches[g].ratio);
  }
  // Eight CTAs whatever the size (64 requests with four tokens each 5.45 us, 5.65 with one CTA; 65k tokens of 300 prompts 11.4,
  // 16 with four and 44 with one), of more threads where lists are long; with 256, 512 and 1024 threads a CTA
  //   requests of 4 tokens, one cache: 64 5.5, 5.7, 6.1 us; 512 6.6, 7.5, 8.2; 1000 7.8, 8.3, 10.9; 2048 12.3, 9.9, 12.1; 4000 25.6, 16.3, 14.9
  //   1000 requests in three caches: 15.0, 13.3, 13.9
  //   60 prompts of 8k tokens in all: 5.0, 5.5, 7.0; 16k 6.4, 5.8, 7.4; 20k 7.4, 7.0, 7.3; 32k 8.7, 7.1, 7.4; 65k 13.6, 9.7, 9.9; 131k 23.2, 15.5, 14.4
  const int cluster = 8, threads = p.B > 2048 || p.T > 32768 ? 1024 : p.B > 512 || p.T > 16384 ? 512 : 256;
  switch (p.num_caches) {
    case 1: return launch_plan<1>(a, cluster, threads, s);
    case 2: return launch_plan<2>(a, cluster, threads, s);
    case 3: return launch_plan<3>(a, cluster, threads, s);
    default: return launch_plan<4>(a, cluster, threads, s);
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
