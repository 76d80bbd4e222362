// Append of new keys and values to paged per-head caches, keys and queries rotated on the way.
//
// One launch, two kinds of CTA.  A cache CTA takes the rows of K or of V that one sequence stores into one
// page for one kv head.  A thread holds up to 4 of their 16-byte chunks in registers, so rows are read once
// although the e4m3 exponent of a (page, head) needs the maximum over all of them before the first code is
// written (more rows than that are read again, from the caches of the first reading).  A query CTA takes one
// token: a thread keeps the cos and sin of its chunk and turns that chunk of head after head, four in flight,
// whose loads go out before the token's position is known.
// The rotation is fp32 with every product and sum rounded (no contraction), so codes and exponents
// are the same whatever kernel or library computes them from the formula.
// Bound by HBM: every row is read once and written once.  11.5k prompt rows of 64 query and 8 kv heads of 128 into e4m3
// (447 MB): 88 us, 5.1 TB/s; 3.6k rows of 20 and 4 heads of 64 (26 MB) into bf16 9.8 us and 32 decode steps (1.25 MB) 6.7, launch latency.
#include "gqa_common.cuh"

namespace dsv4 {

static __device__ unsigned int g_flags_ga = 0;

namespace gqa {

struct Rope {
  const float* cos_sin;
  int first, half, halves;
};

// cos and sin of chunk c (dims 8c .. 8c + 7) of a row at position pos: 4 pairs (GPT-J), or with halves the 8 dims'
// own, both in registers; kind: 0 the chunk is not turned, 1 GPT-J pairs, 2 / 3 the lower / upper half.
struct Turn {
  float co[8], si[8];
  int kind;
};

template <int N>
__device__ __forceinline__ void load_turn(Turn& tr, const float* cs, int half) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {  // (16-byte aligned: rope_dim is a multiple of 16, dims come by 8)
    const float4 a = __ldg(reinterpret_cast<const float4*>(cs + i)), b = __ldg(reinterpret_cast<const float4*>(cs + half + i));
    tr.co[i] = a.x, tr.co[i + 1] = a.y, tr.co[i + 2] = a.z, tr.co[i + 3] = a.w;
    tr.si[i] = b.x, tr.si[i + 1] = b.y, tr.si[i + 2] = b.z, tr.si[i + 3] = b.w;
  }
}

__device__ __forceinline__ void turn_of(const Rope& r, int c, int64_t pos, bool live, Turn& tr) {
  const int d0 = 8 * c - r.first;  // the chunk's first dim inside the rotated range
  tr.kind = 0;
  if (r.cos_sin == nullptr || !live || d0 < 0 || d0 >= 2 * r.half) return;
  const float* row = r.cos_sin + pos * (2 * r.half);
  if (!r.halves) {
    tr.kind = 1;
    load_turn<4>(tr, row + d0 / 2, r.half);
  } else {
    tr.kind = d0 < r.half ? 2 : 3;
    load_turn<8>(tr, row + (d0 < r.half ? d0 : d0 - r.half), r.half);
  }
}

// The chunk's bf16 values `raw`, turned.  With halves, the partner dims are in chunk c +- half / 8 of the same
// row, which another lane of the warp holds (CPR lanes hold one row); every lane of the warp calls this.
template <int CPR>
__device__ __forceinline__ void rotate_chunk(const Rope& r, const Turn& tr, const uint4& raw, int c, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (r.cos_sin == nullptr) return;
  if (!r.halves) {
    if (tr.kind == 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, tr.co[i]), __fmul_rn(b, tr.si[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, tr.co[i]), __fmul_rn(a, tr.si[i]));
    }
    return;
  }
  const int lane = threadIdx.x & 31, row0 = lane & ~(CPR - 1);
  const int src = tr.kind ? row0 + c + (tr.kind == 2 ? r.half / 8 : -(r.half / 8)) : lane;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], src);
  if (tr.kind == 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __uint_as_float(i & 1 ? o[i >> 1] & 0xFFFF0000u : o[i >> 1] << 16);
    x[i] = tr.kind == 2 ? __fsub_rn(__fmul_rn(x[i], tr.co[i]), __fmul_rn(y, tr.si[i]))
                        : __fadd_rn(__fmul_rn(x[i], tr.co[i]), __fmul_rn(y, tr.si[i]));
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&x)[8]) {
  return make_uint4(float2_to_bf16x2_bits(x[0], x[1]), float2_to_bf16x2_bits(x[2], x[3]),
                    float2_to_bf16x2_bits(x[4], x[5]), float2_to_bf16x2_bits(x[6], x[7]));
}

// Exponent of a (page, head) whose largest stored magnitude is amax: -127 for 0, so that a later
// append's exponent always wins.
__device__ __forceinline__ int page_exponent(float amax) { return amax == 0.f ? -127 : ue8m0_exponent(amax); }

// Queries: one token a CTA.
template <int D, int THREADS>
__device__ __forceinline__ void rotate_queries(const dsv4_gqa_append_params& p, const Rope& rope, int t) {
  constexpr int CPR = D / 8, HPI = THREADS / CPR;  // heads the CTA turns at once
  const int lane = threadIdx.x & 31, c = threadIdx.x % CPR, hl = threadIdx.x / CPR;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)t * p.q_token_stride + 8 * c;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.q_out) + (int64_t)t * p.q_out_token_stride + 8 * c;
  uint4 raw[4];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = h0 + i * HPI + hl;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (h < p.q_heads) raw[i] = *reinterpret_cast<const uint4*>(q + (int64_t)h * p.q_head_stride);
    }
  };
  load(0);
  // the token's sequence: the last b with q_start[b] <= t (32 probes a step)
  int lo = 0, hi = p.B;  // the answer is in [lo, hi)
  if (p.q_start[0] > t) return;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && p.q_start[at] <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const Seq s = sequence(p.q_start, p.kv_len, lo, p.T, p.max_q_len, p.cos_sin ? p.max_pos : MAX_ROWS);
  if (!s.ok || t >= s.t0 + s.n) return;  // padding behind the last sequence, or a skipped sequence
  Turn tr;
  turn_of(rope, c, s.kv - s.n + (t - s.t0), true, tr);
  for (int h0 = 0; h0 < p.q_heads; h0 += 4 * HPI) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = h0 + i * HPI + hl;
      float x[8];
      rotate_chunk<CPR>(rope, tr, raw[i], c, x);
      if (h < p.q_heads) *reinterpret_cast<uint4*>(o + (int64_t)h * p.q_out_head_stride) = pack_bf16(x);
    }
  }
}

// The queries of a long append, after append_kernel on the stream: starts once that one's CTAs have all started
// (which were let go when the kernels before had finished), and ends after it.
template <int D>
__global__ void __launch_bounds__(256, 4) append_queries_kernel(dsv4_gqa_append_params p) {
  pdl_start(true);
  Rope rope;
  rope.cos_sin = p.cos_sin;
  rope.first = p.rope_first;
  rope.half = p.rope_dim / 2;
  rope.halves = p.rope_halves;
  rotate_queries<D, 256>(p, rope, blockIdx.x);
  pdl_wait();
}

template <int D, bool E4M3, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 64 ? 8 : E4M3 ? 2 : 3)
    append_kernel(dsv4_gqa_append_params p, int q_ctas, int pages_per_seq) {
  constexpr int CPR = D / 8;       // 16-byte chunks of a bf16 row
  constexpr int RPI = THREADS / CPR, NR = 4;
  pdl_wait();
  pdl_launch_dependents();
  Rope rope;
  rope.cos_sin = p.cos_sin;
  rope.first = p.rope_first;
  rope.half = p.rope_dim / 2;
  rope.halves = p.rope_halves;
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < q_ctas) {
    rotate_queries<D, THREADS>(p, rope, blockIdx.x);
    return;
  }
  const int item = blockIdx.x - q_ctas;
  const bool is_v = item & 1;
  const int h = (item >> 1) % p.kv_heads, u = (item >> 1) / p.kv_heads;
  const int b = u / pages_per_seq, slot = u % pages_per_seq;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.cos_sin ? p.max_pos : MAX_ROWS);
  if (!s.ok) {
    if (slot == 0 && h == 0 && tid == 0) atomicOr(&g_flags_ga, FLAG_PAGE);
    return;
  }
  const int p0 = s.kv - s.n, lp = p0 / p.page_size + slot, first = lp * p.page_size;
  const int lo = max(first, p0), hi = min(first + p.page_size, s.kv);
  if (lo >= hi) return;
  const int page = lp < p.max_pages_per_seq ? p.block_table[(int64_t)b * p.max_pages_per_seq + lp] : -1;
  if (is_v) rope.cos_sin = nullptr;
  const int c = tid % CPR, r0 = tid / CPR;
  const int64_t tstride = is_v ? p.v_token_stride : p.k_token_stride;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) +
                             (int64_t)h * (is_v ? p.v_head_stride : p.k_head_stride) + 8 * c;
  uint4 raw[NR];
  auto load = [&](int from) {  // NR chunks of this thread, from row `from` on
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = from + r0 + i * RPI;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (row < hi) raw[i] = *reinterpret_cast<const uint4*>(src + (int64_t)(s.t0 + (row - p0)) * tstride);
    }
  };
  auto turned = [&](int from, int i, float (&x)[8]) {
    const int row = from + r0 + i * RPI;
    Turn tr;
    turn_of(rope, c, row, row < hi, tr);
    rotate_chunk<CPR>(rope, tr, raw[i], c, x);
  };
  load(lo);
  if (page < 0 || page >= p.num_pages) {
    if (h == 0 && tid == 0 && !is_v) atomicOr(&g_flags_ga, FLAG_PAGE);
    return;
  }
  const int64_t rstride = is_v ? p.v_row_stride : p.k_row_stride;
  const int64_t base = (int64_t)page * (is_v ? p.v_page_stride : p.k_page_stride) +
                       (int64_t)h * (is_v ? p.v_cache_head_stride : p.k_cache_head_stride);
  if (!E4M3) {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + base + 8 * c;
    for (int from = lo; from < hi; from += NR * RPI) {
      if (from > lo) load(from);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int row = from + r0 + i * RPI;
        float x[8];
        turned(from, i, x);
        if (row < hi) *reinterpret_cast<uint4*>(dst + (int64_t)(row - first) * rstride) = pack_bf16(x);
      }
    }
    return;
  }
  uint8_t* ex = (is_v ? p.v_exp : p.k_exp) + (int64_t)page * p.kv_heads + h;
  const int old = lo > first ? (int)*ex - 127 : 0;
  float x[NR][8], amax = 0.f;
  const bool once = hi - lo <= NR * RPI;  // everything stays in registers
  for (int from = lo; from < hi; from += NR * RPI) {
    if (from > lo) load(from);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      turned(from, i, x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[i][j]));
    }
  }
  __shared__ float red[32];
  amax = warp_max(amax);
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
  int e = page_exponent(amax);
  uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + base;
  if (lo > first) {
    e = max(e, old);
    const int d = e - old;
    if (d > 0) {  // rows stored earlier, re-encoded for the larger exponent
      const float f = d < 64 ? exp2_neg_int(d) : 0.f;  // (code magnitudes lie in [2^-9, 448]: 0 from 2^-64 on)
      for (int y = tid; y < (lo - first) * (D / 4); y += THREADS) {
        uint32_t* a = reinterpret_cast<uint32_t*>(dst + (int64_t)(y / (D / 4)) * rstride) + y % (D / 4);
        const uint32_t w = *a;
        const float2 g0 = e4m3x2_to_float2((uint16_t)(w & 0xFFFFu)), g1 = e4m3x2_to_float2((uint16_t)(w >> 16));
        *a = (uint32_t)float2_to_e4m3x2(g0.x * f, g0.y * f) | ((uint32_t)float2_to_e4m3x2(g1.x * f, g1.y * f) << 16);
      }
    }
  }
  if (tid == 0) *ex = (uint8_t)(e + 127);  // (every thread has read the old one: the barrier above)
  const float f = exp2_neg_int(e);
  for (int from = lo; from < hi; from += NR * RPI) {
    if (!once) load(from);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (!once) turned(from, i, x[i]);
      const int row = from + r0 + i * RPI;
      uint32_t o[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        o[j] = (uint32_t)float2_to_e4m3x2(x[i][4 * j] * f, x[i][4 * j + 1] * f) |
               ((uint32_t)float2_to_e4m3x2(x[i][4 * j + 2] * f, x[i][4 * j + 3] * f) << 16);
      if (row < hi) *reinterpret_cast<uint2*>(dst + (int64_t)(row - first) * rstride + 8 * c) = make_uint2(o[0], o[1]);
    }
  }
}

template <int D, int THREADS>
cudaError_t launch_append(const dsv4_gqa_append_params& p, dim3 grid, int q_ctas, int pages, cudaStream_t s) {
  return p.cache_dtype == DSV4_E4M3_PAGE
             ? launch_pdl(append_kernel<D, true, THREADS>, grid, dim3(THREADS), 0, s, true, p, q_ctas, pages)
             : launch_pdl(append_kernel<D, false, THREADS>, grid, dim3(THREADS), 0, s, true, p, q_ctas, pages);
}

}  // namespace gqa

cudaError_t launch_gqa_append(const dsv4_gqa_append_params& p, cudaStream_t s) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  const int max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  const int pages = (max_n + p.page_size - 2) / p.page_size + 1;  // pages a sequence's new rows can touch
  const int q_ctas = p.q != nullptr ? p.T : 0;
  // Few rows a page (decode steps, small pages): two warps hold them, and their barrier and idle lanes cost less than
  // eight's (32 decode steps 6.7 us, 8.4 with eight; prompts into bf16 pages of 16 rows 9.8 and 25).
  const int rows = max_n < p.page_size ? max_n : p.page_size;
  // There the queries ride along; else they are a second kernel, whose CTAs need half the registers (105 us for 88).
  const bool small = rows * p.head_dim / 8 <= 64 * 4;
  const int64_t grid = 2 * (int64_t)p.B * pages * p.kv_heads + (small ? q_ctas : 0);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)grid);
  if (small)
    return p.head_dim == 128 ? gqa::launch_append<128, 64>(p, g, q_ctas, pages, s)
                             : gqa::launch_append<64, 64>(p, g, q_ctas, pages, s);
  const cudaError_t e = p.head_dim == 128 ? gqa::launch_append<128, 256>(p, g, 0, pages, s)
                                          : gqa::launch_append<64, 256>(p, g, 0, pages, s);
  if (e != cudaSuccess || q_ctas == 0) return e;
  return p.head_dim == 128 ? launch_pdl(gqa::append_queries_kernel<128>, dim3(q_ctas), dim3(256), 0, s, true, p)
                           : launch_pdl(gqa::append_queries_kernel<64>, dim3(q_ctas), dim3(256), 0, s, true, p);
}

cudaError_t read_flags_gqa_append(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_ga, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_ga, &z, sizeof(z));
}

}  // namespace dsv4
