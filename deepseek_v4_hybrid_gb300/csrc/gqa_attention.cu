// Grouped-query attention of new tokens over paged per-head caches.
//
// Simple form: one warp per (token, query head), the row's dims spread over the lanes, fp32 online
// softmax over the visible rows.
#include "gqa_attention.cuh"

namespace dsv4 {

static __device__ unsigned int g_flags_gq = 0;

namespace gqa {

template <int D>
__global__ void __launch_bounds__(128) attention_simple(dsv4_gqa_attention_params p) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(unit % p.q_heads), t = (int)(unit / p.q_heads);
  if (t >= p.T) return;
  int b = 0;
  while (b + 1 < p.B && p.q_start[b + 1] <= t) ++b;
  const Seq s = sequence(p.q_start, p.kv_len, b, p.T, p.max_q_len, p.max_kv_len);
  if (!s.ok) {
    if (lane == 0 && h == 0) atomicOr(&g_flags_gq, FLAG_PAGE);
    return;
  }
  if (t < s.t0 || t >= s.t0 + s.n) return;
  const int pos = s.kv - s.n + (t - s.t0), hk = h / (p.q_heads / p.kv_heads);
  const int2 vis = visible_rows(p, b, t, pos, s.kv);
  float q[E], o[E];
  const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)t * p.q_token_stride + (int64_t)h * p.q_head_stride;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(qp[lane + 32 * i]);
    o[i] = 0.f;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = p.sink ? p.sink[h] : -INFINITY, l = m > -INFINITY ? 1.f : 0.f;
  for (int j = vis.x; j < vis.y; ++j) {
    const int lp = j / p.page_size, off = j % p.page_size;
    const int page = lp < p.max_pages_per_seq ? p.block_table[(int64_t)b * p.max_pages_per_seq + lp] : -1;
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(&g_flags_gq, FLAG_PAGE);
      continue;
    }
    const int64_t ko = (int64_t)page * p.k_page_stride + (int64_t)hk * p.k_cache_head_stride + (int64_t)off * p.k_row_stride;
    const int64_t vo = (int64_t)page * p.v_page_stride + (int64_t)hk * p.v_cache_head_stride + (int64_t)off * p.v_row_stride;
    float k[E], v[E];
    if (p.cache_dtype == DSV4_BF16) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        k[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.k_cache)[ko + lane + 32 * i]);
        v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v_cache)[vo + lane + 32 * i]);
      }
    } else {
      const float fk = ue8m0_scale(p.k_exp[(int64_t)page * p.kv_heads + hk]);
      const float fv = ue8m0_scale(p.v_exp[(int64_t)page * p.kv_heads + hk]);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        k[i] = e4m3x2_to_float2(reinterpret_cast<const uint8_t*>(p.k_cache)[ko + lane + 32 * i]).x * fk;
        v[i] = e4m3x2_to_float2(reinterpret_cast<const uint8_t*>(p.v_cache)[vo + lane + 32 * i]).x * fv;
      }
    }
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) z = fmaf(q[i], k[i], z);
    z = warp_sum(z) * p.softmax_scale;
    if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
    z -= slope * (float)abs(pos - j);
    const float mn = fmaxf(m, z), f = expf(m - mn), w = expf(z - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * f + w * v[i];
    m = mn;
  }
  const int64_t row = (int64_t)t * p.q_heads + h;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (p.out_dtype == DSV4_F32)
      reinterpret_cast<float*>(p.out)[row * D + lane + 32 * i] = o[i] * inv;
    else
      reinterpret_cast<__nv_bfloat16*>(p.out)[row * D + lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
  }
  if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace gqa

// Up to 32 rows of (token, head) a kv head and sequence: the streaming kernel.
static bool use_decode(const dsv4_gqa_attention_params& p) {
  const int64_t max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  return max_n * (p.q_heads / p.kv_heads) <= 32;
}

size_t gqa_attention_workspace(const dsv4_gqa_attention_params& p) {
  if (p.T == 0 || p.B == 0) return 256;
  return use_decode(p) ? gqa::decode_workspace(p) : 256;
}

cudaError_t launch_gqa_attention(const dsv4_gqa_attention_params& p, cudaStream_t s) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  if (use_decode(p)) return gqa::launch_decode(p, s);
  const int64_t units = (int64_t)p.T * p.q_heads;
  const dim3 grid((unsigned)((units + 3) / 4));
  return p.head_dim == 128 ? launch_pdl(gqa::attention_simple<128>, grid, dim3(128), 0, s, true, p)
                           : launch_pdl(gqa::attention_simple<64>, grid, dim3(128), 0, s, true, p);
}

cudaError_t read_flags_gqa_attention(uint32_t* f) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_flags_gq, sizeof(v));
  if (e != cudaSuccess) return e;
  *f |= v;
  return cudaMemcpyToSymbol(g_flags_gq, &z, sizeof(z));
}

}  // namespace dsv4
