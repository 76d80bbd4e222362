// Pieces shared by the grouped-query attention kernels: which rows a token sees, and how a row's sums
// become its output.
#pragma once

#include "gqa_common.cuh"
#include "tc_ptx.cuh"

namespace dsv4 {
namespace gqa {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

// First and one-past-last visible row of token t at position pos (the visible rows are contiguous).
__device__ __forceinline__ int2 visible_rows(const dsv4_gqa_attention_params& p, int b, int t, int pos, int kv) {
  int lo = p.kv_start ? max(0, p.kv_start[t]) : 0, hi = kv;
  if (p.causal) {
    hi = pos + 1;
    if (p.prefix_len) hi = max(hi, min(kv, p.prefix_len[b]));
  }
  if (p.window > 0) lo = max(lo, pos - p.window + 1);
  return make_int2(lo, hi);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(z / cap) with rcap2 = 2 log2(e) / cap: tanh x = 1 - 2 / (1 + e^2x), off by less than 2^-20 cap.
__device__ __forceinline__ float cap_logit(float z, float cap, float rcap2) {
  return cap - 2.f * cap * rcp_approx(1.f + tc::ex2_approx(z * rcap2));
}

// A row's sums: m the reference (log2 units) that its weights are taken against, l their sum.  Returns the factor
// of the output's sum, writes lse when `write` is set.
__device__ __forceinline__ float finish_scale(const dsv4_gqa_attention_params& p, int64_t row, int head, float m, float l,
                                              bool write) {
  const float sink = p.sink ? p.sink[head] * LOG2E : -INFINITY;
  const float mf = fmaxf(m, sink);
  const float f = m > -INFINITY ? tc::ex2_approx(m - mf) : 0.f;
  float L = l * f;
  if (sink > -INFINITY) L += tc::ex2_approx(sink - mf);
  if (write && p.lse) p.lse[row] = mf > -INFINITY ? (mf + __log2f(L)) * LN2 : -INFINITY;
  return m > -INFINITY ? f * rcp_approx(L) : 0.f;
}

// Stores 4 consecutive dims of an output row.
template <int D>
__device__ __forceinline__ void store4(const dsv4_gqa_attention_params& p, int64_t row, int d4, float4 v) {
  if (p.out_dtype == DSV4_F32)
    reinterpret_cast<float4*>(p.out)[row * (D / 4) + d4] = v;
  else
    reinterpret_cast<uint2*>(p.out)[row * (D / 4) + d4] =
        make_uint2(float2_to_bf16x2_bits(v.x, v.y), float2_to_bf16x2_bits(v.z, v.w));
}

size_t decode_workspace(const dsv4_gqa_attention_params& p);
size_t prefill_workspace(const dsv4_gqa_attention_params& p);
cudaError_t launch_prefill(const dsv4_gqa_attention_params& p, cudaStream_t s);
cudaError_t launch_decode(const dsv4_gqa_attention_params& p, cudaStream_t s);

}  // namespace gqa
}  // namespace dsv4
