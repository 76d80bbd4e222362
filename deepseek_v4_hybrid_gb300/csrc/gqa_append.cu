// Append of new keys and values to paged per-head caches, keys and queries rotated on the way.
//
// One launch, two kinds of CTA.  A cache CTA takes the rows that one sequence stores into one page for
// one kv head, keys and values both: a thread holds up to NR 16-byte chunks of each in registers, so the
// rows are read once although the e4m3 exponent of a (page, head) needs the maximum over all of them
// before the first code is written.  A query CTA takes one token: a thread keeps the cos and sin of its
// chunk in registers and turns that chunk of head after head.
// The rotation is fp32 with every product and sum rounded (no contraction), so codes and exponents
// are the same whatever kernel or library computes them from the formula.
// Bound by HBM: every row is read once and written once.
#include "gqa_common.cuh"

namespace dsv4 {

static __device__ unsigned int g_flags_ga = 0;

namespace gqa {

constexpr int Q_THREADS = 256;

struct Rope {
  const float* cos_sin;
  int first, half, halves;
};

// Chunk c (dims 8c .. 8c + 7) of a row at position pos, whose bf16 values are `raw`, rotated.  With
// halves, the partner dims are in chunk c +- half / 8 of the same row, which another lane of the warp
// holds (`cpr` lanes hold one row); every lane of the warp calls this.
template <int CPR>
__device__ __forceinline__ void rotate_chunk(const Rope& r, const uint4& raw, int c, int64_t pos, bool live,
                                             float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (r.cos_sin == nullptr) return;
  const int d0 = 8 * c - r.first;  // the chunk's first dim inside the rotated range
  const bool in = live && d0 >= 0 && d0 < 2 * r.half;
  if (!r.halves) {
    if (!in) return;
    const float* cs = r.cos_sin + pos * (2 * r.half) + d0 / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float co = __ldg(cs + i), si = __ldg(cs + r.half + i), a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si));
    }
    return;
  }
  const bool low = d0 < r.half;
  const int lane = threadIdx.x & 31, row0 = lane & ~(CPR - 1);
  const int src = in ? row0 + c + (low ? r.half / 8 : -(r.half / 8)) : lane;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], src);
  if (!in) return;
  const float* cs = r.cos_sin + pos * (2 * r.half) + (low ? d0 : d0 - r.half);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float co = __ldg(cs + i), si = __ldg(cs + r.half + i);
    const float y = __uint_as_float(i & 1 ? o[i >> 1] & 0xFFFF0000u : o[i >> 1] << 16);
    x[i] = low ? __fsub_rn(__fmul_rn(x[i], co), __fmul_rn(y, si)) : __fadd_rn(__fmul_rn(x[i], co), __fmul_rn(y, si));
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
template <int D>
__device__ __forceinline__ void rotate_queries(const dsv4_gqa_append_params& p, const Rope& rope, int t) {
  constexpr int CPR = D / 8;
  // the token's sequence: the last b with q_start[b] <= t (32 probes a step)
  const int lane = threadIdx.x & 31;
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
  const Seq s = sequence(p.q_start, p.kv_len, lo, p.T, p.max_q_len, p.cos_sin ? p.max_pos : -1);
  if (!s.ok || t >= s.t0 + s.n) return;  // padding behind the last sequence, or a skipped sequence
  const int64_t pos = s.kv - s.n + (t - s.t0);
  const int c = threadIdx.x % CPR;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)t * p.q_token_stride + 8 * c;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.q_out) + (int64_t)t * p.q_out_token_stride + 8 * c;
  for (int h0 = 0; h0 < p.q_heads; h0 += Q_THREADS / CPR) {
    const int h = h0 + threadIdx.x / CPR;
    const bool live = h < p.q_heads;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(q + (int64_t)h * p.q_head_stride);
    float x[8];
    rotate_chunk<CPR>(rope, raw, c, pos, live, x);
    if (live) *reinterpret_cast<uint4*>(o + (int64_t)h * p.q_out_head_stride) = pack_bf16(x);
  }
}

template <int D, int NR, bool E4M3>
__global__ void __launch_bounds__(1024) append_kernel(dsv4_gqa_append_params p, int q_ctas, int pages_per_seq) {
  constexpr int CPR = D / 8;  // 16-byte chunks of a bf16 row
  pdl_wait();
  pdl_launch_dependents();
  Rope rope;
  rope.cos_sin = p.cos_sin;
  rope.first = p.rope_first;
  rope.half = p.rope_dim / 2;
  rope.halves = p.rope_halves;
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < q_ctas) {
    if (tid < Q_THREADS) rotate_queries<D>(p, rope, blockIdx.x);
    return;
  }
  const int item = blockIdx.x - q_ctas;
  const int h = item % p.kv_heads, u = item / p.kv_heads;
  const int b = u / pages_per_seq, slot = u % pages_per_seq;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.cos_sin ? p.max_pos : -1);
  if (!s.ok) {
    if (slot == 0 && h == 0 && tid == 0) atomicOr(&g_flags_ga, FLAG_PAGE);
    return;
  }
  const int p0 = s.kv - s.n, lp = p0 / p.page_size + slot, first = lp * p.page_size;
  const int lo = max(first, p0), hi = min(first + p.page_size, s.kv);
  if (lo >= hi) return;
  const int page = lp < p.max_pages_per_seq ? p.block_table[(int64_t)b * p.max_pages_per_seq + lp] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (h == 0 && tid == 0) atomicOr(&g_flags_ga, FLAG_PAGE);
    return;
  }
  const int64_t eslot = (int64_t)page * p.kv_heads + h;
  int old_k = 0, old_v = 0;
  if (E4M3 && lo > first) {
    old_k = (int)p.k_exp[eslot] - 127;
    old_v = (int)p.v_exp[eslot] - 127;
  }
  const int c = tid % CPR, r0 = tid / CPR, rstep = blockDim.x / CPR;
  const __nv_bfloat16* kn = reinterpret_cast<const __nv_bfloat16*>(p.k_new) + (int64_t)h * p.k_head_stride + 8 * c;
  const __nv_bfloat16* vn = reinterpret_cast<const __nv_bfloat16*>(p.v_new) + (int64_t)h * p.v_head_stride + 8 * c;
  uint4 kraw[NR], vraw[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = lo + r0 + i * rstep;
    kraw[i] = vraw[i] = make_uint4(0, 0, 0, 0);
    if (row < hi) {
      const int64_t t = s.t0 + (row - p0);
      kraw[i] = *reinterpret_cast<const uint4*>(kn + t * p.k_token_stride);
      vraw[i] = *reinterpret_cast<const uint4*>(vn + t * p.v_token_stride);
    }
  }
  if (!E4M3) {
    __nv_bfloat16* kc = reinterpret_cast<__nv_bfloat16*>(p.k_cache) + (int64_t)page * p.k_page_stride +
                        (int64_t)h * p.k_cache_head_stride + 8 * c;
    __nv_bfloat16* vc = reinterpret_cast<__nv_bfloat16*>(p.v_cache) + (int64_t)page * p.v_page_stride +
                        (int64_t)h * p.v_cache_head_stride + 8 * c;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = lo + r0 + i * rstep;
      float x[8];
      rotate_chunk<CPR>(rope, kraw[i], c, row, row < hi, x);
      if (row < hi) {
        *reinterpret_cast<uint4*>(kc + (int64_t)(row - first) * p.k_row_stride) = pack_bf16(x);
        *reinterpret_cast<uint4*>(vc + (int64_t)(row - first) * p.v_row_stride) = vraw[i];
      }
    }
    return;
  }
  float kx[NR][8], kmax = 0.f, vmax = 0.f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = lo + r0 + i * rstep;
    rotate_chunk<CPR>(rope, kraw[i], c, row, row < hi, kx[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) kmax = fmaxf(kmax, fabsf(kx[i][j]));
    const uint32_t w[4] = {vraw[i].x, vraw[i].y, vraw[i].z, vraw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      vmax = fmaxf(vmax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
  }
  __shared__ float red[2][32];
  kmax = warp_max(kmax);
  vmax = warp_max(vmax);
  if ((tid & 31) == 0) {
    red[0][tid >> 5] = kmax;
    red[1][tid >> 5] = vmax;
  }
  __syncthreads();
  const int nw = blockDim.x / 32, lane = tid & 31;
  kmax = warp_max(lane < nw ? red[0][lane] : 0.f);
  vmax = warp_max(lane < nw ? red[1][lane] : 0.f);
  int ek = page_exponent(kmax), ev = page_exponent(vmax);
  uint8_t* kc = reinterpret_cast<uint8_t*>(p.k_cache) + (int64_t)page * p.k_page_stride +
                (int64_t)h * p.k_cache_head_stride;
  uint8_t* vc = reinterpret_cast<uint8_t*>(p.v_cache) + (int64_t)page * p.v_page_stride +
                (int64_t)h * p.v_cache_head_stride;
  if (lo > first) {
    ek = max(ek, old_k);
    ev = max(ev, old_v);
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {  // rows stored earlier, re-encoded where the exponent grew
      const int d = kv ? ev - old_v : ek - old_k;
      if (d == 0) continue;
      const float f = d < 64 ? exp2_neg_int(d) : 0.f;  // (code magnitudes lie in [2^-9, 448]: 0 from 2^-64 on)
      uint8_t* base = kv ? vc : kc;
      const int64_t rs = kv ? p.v_row_stride : p.k_row_stride;
      for (int x = tid; x < (lo - first) * (D / 4); x += blockDim.x) {
        uint32_t* a = reinterpret_cast<uint32_t*>(base + (int64_t)(x / (D / 4)) * rs) + x % (D / 4);
        const uint32_t w = *a;
        const float2 g0 = e4m3x2_to_float2((uint16_t)(w & 0xFFFFu)), g1 = e4m3x2_to_float2((uint16_t)(w >> 16));
        *a = (uint32_t)float2_to_e4m3x2(g0.x * f, g0.y * f) | ((uint32_t)float2_to_e4m3x2(g1.x * f, g1.y * f) << 16);
      }
    }
  }
  if (tid == 0) {
    p.k_exp[eslot] = (uint8_t)(ek + 127);
    p.v_exp[eslot] = (uint8_t)(ev + 127);
  }
  const float fk = exp2_neg_int(ek), fv = exp2_neg_int(ev);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = lo + r0 + i * rstep;
    if (row >= hi) continue;
    uint32_t ko[2], vo[2];
    const uint32_t w[4] = {vraw[i].x, vraw[i].y, vraw[i].z, vraw[i].w};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      ko[j] = (uint32_t)float2_to_e4m3x2(kx[i][4 * j] * fk, kx[i][4 * j + 1] * fk) |
              ((uint32_t)float2_to_e4m3x2(kx[i][4 * j + 2] * fk, kx[i][4 * j + 3] * fk) << 16);
      vo[j] = (uint32_t)float2_to_e4m3x2(__uint_as_float(w[2 * j] << 16) * fv,
                                         __uint_as_float(w[2 * j] & 0xFFFF0000u) * fv) |
              ((uint32_t)float2_to_e4m3x2(__uint_as_float(w[2 * j + 1] << 16) * fv,
                                          __uint_as_float(w[2 * j + 1] & 0xFFFF0000u) * fv)
               << 16);
    }
    *reinterpret_cast<uint2*>(kc + (int64_t)(row - first) * p.k_row_stride + 8 * c) = make_uint2(ko[0], ko[1]);
    *reinterpret_cast<uint2*>(vc + (int64_t)(row - first) * p.v_row_stride + 8 * c) = make_uint2(vo[0], vo[1]);
  }
}

template <int D, int NR>
cudaError_t launch_append(const dsv4_gqa_append_params& p, dim3 grid, int threads, int q_ctas, int pages,
                          cudaStream_t s) {
  return p.cache_dtype == DSV4_E4M3_PAGE
             ? launch_pdl(append_kernel<D, NR, true>, grid, dim3(threads), 0, s, true, p, q_ctas, pages)
             : launch_pdl(append_kernel<D, NR, false>, grid, dim3(threads), 0, s, true, p, q_ctas, pages);
}

}  // namespace gqa

cudaError_t launch_gqa_append(const dsv4_gqa_append_params& p, cudaStream_t s) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  const int max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  const int pages = (max_n + p.page_size - 2) / p.page_size + 1;  // pages a sequence's new rows can touch
  const int q_ctas = p.q != nullptr ? p.T : 0;
  const int64_t grid = (int64_t)q_ctas + (int64_t)p.B * pages * p.kv_heads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const int chunks = p.page_size * p.head_dim / 8;  // of a whole page: NR a thread
  const int nr = chunks <= 256 ? 1 : chunks <= 512 ? 2 : 4;
  const int threads = chunks / nr < 256 ? 256 : chunks / nr;
  const dim3 g((unsigned)grid);
  if (p.head_dim == 128) {
    if (nr == 1) return gqa::launch_append<128, 1>(p, g, threads, q_ctas, pages, s);
    if (nr == 2) return gqa::launch_append<128, 2>(p, g, threads, q_ctas, pages, s);
    return gqa::launch_append<128, 4>(p, g, threads, q_ctas, pages, s);
  }
  if (nr == 1) return gqa::launch_append<64, 1>(p, g, threads, q_ctas, pages, s);
  if (nr == 2) return gqa::launch_append<64, 2>(p, g, threads, q_ctas, pages, s);
  return gqa::launch_append<64, 4>(p, g, threads, q_ctas, pages, s);
}

cudaError_t read_flags_gqa_append(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_ga, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_ga, &z, sizeof(z));
}

}  // namespace dsv4
