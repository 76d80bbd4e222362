// Rotary positions: rows turned by their tokens' positions, and the cos / sin tables.
//
// An angle is position * f_i / (2 pi) turns.  With the frequency as a 64-bit binary fraction of a turn, the product
// modulo 2^64 is the angle reduced to one turn, exactly, for every position: one integer product in the place of
// a reduction by 2 pi in wider floating point.  Its 64 bits are split into the nearest quarter turn and a rest that
// becomes an fp32 number of half turns for sincospi, so that a sine or cosine near 0 keeps its relative accuracy.
//
// A thread owns 8 dims (or 8 + 8 partner dims with halves) of a token's heads: it computes their cos and sin once and
// turns that chunk of head after head, so nothing is shared and nothing waits but the loads.
#include "loop_common.cuh"

namespace dsv4 {
namespace loop {

// cos and sin of position p under a frequency, times scale.
__device__ __forceinline__ void turn(uint32_t p, uint64_t freq, float scale, float& co, float& si) {
  const uint64_t t = p * freq, quadrant = (t + (1ull << 61)) >> 62;
  float c, s;
  sincospif(__ll2float_rn((long long)(t - (quadrant << 62))) * 0x1p-63f, &s, &c);  // of [-1/4, 1/4]
  const float a = quadrant & 1 ? s : c, b = quadrant & 1 ? c : s;
  co = (quadrant + 1) & 2 ? -scale * a : scale * a;
  si = quadrant & 2 ? -scale * b : scale * b;
}

template <bool F32>
struct Chunk;  // 8 elements

template <>
struct Chunk<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + at);
    a = p[0], b = p[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
    p[0] = a, p[1] = b;
  }
};

template <>
struct Chunk<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    a = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + at);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_uint4(float2_to_bf16x2_bits(v[0], v[1]), float2_to_bf16x2_bits(v[2], v[3]),
                   float2_to_bf16x2_bits(v[4], v[5]), float2_to_bf16x2_bits(v[6], v[7]));
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + at) = a;
  }
};

// blockDim = (items of a head, heads at once, tokens).  Item c < pairs turns a chunk (halves: and its partner), the
// others copy one.
template <bool F32, bool HALVES>
__global__ void __launch_bounds__(256) rope_kernel(const dsv4_rope_params p, int pairs) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = (int64_t)blockIdx.x * blockDim.z + threadIdx.z;
  if (t >= p.T) return;
  const int pos = p.positions[t];
  if (pos < 0) return;
  const int c = threadIdx.x, half = p.rope_dim / 2;
  const bool turned = c < pairs;
  int d = p.rope_first + 8 * c;  // first dim of the chunk
  if (!turned) {
    d = 8 * (c - pairs);
    if (d >= p.rope_first) d += p.rope_dim;
  }
  constexpr int NP = HALVES ? 8 : 4;
  float co[NP], si[NP];
  if (turned) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      turn((uint32_t)pos, p.freqs[NP * c + i], p.scale, co[i], si[i]);
      if (p.inverse) si[i] = -si[i];
    }
  }
  const int all = p.heads + (p.x2 ? p.heads2 : 0);
  for (int h = threadIdx.y; h < all; h += blockDim.y) {
    const bool second = h >= p.heads;
    const int hh = second ? h - p.heads : h;
    const void* x = second ? p.x2 : p.x;
    void* y = second ? p.y2 : p.y;
    const int64_t from = t * (second ? p.x2_token_stride : p.x_token_stride) +
                         hh * (second ? p.x2_head_stride : p.x_head_stride) + d;
    const int64_t to = t * (second ? p.y2_token_stride : p.y_token_stride) +
                       hh * (second ? p.y2_head_stride : p.y_head_stride) + d;
    Chunk<F32> u, w;
    u.load(x, from);
    if (turned) {
      float a[8], b[8];
      u.get(a);
      if (HALVES) {
        w.load(x, from + half);
        w.get(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a0 = a[i], b0 = b[i];
          a[i] = a0 * co[i % NP] - b0 * si[i % NP];
          b[i] = b0 * co[i % NP] + a0 * si[i % NP];
        }
        w.set(b);
        w.store(y, to + half);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = a[2 * i], b0 = a[2 * i + 1];
          a[2 * i] = a0 * co[i] - b0 * si[i];
          a[2 * i + 1] = b0 * co[i] + a0 * si[i];
        }
      }
      u.set(a);
    }
    u.store(y, to);
  }
}

// Four pairs of a row a thread.
__global__ void __launch_bounds__(256) rope_table_kernel(const dsv4_rope_table_params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int half = p.rope_dim / 2, quads = half / 4;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (at >= (int64_t)p.rows * quads) return;
  const int64_t row = at / quads;
  const int q = (int)(at - row * quads);
  float co[4], si[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) turn((uint32_t)(p.first_position + row), p.freqs[4 * q + i], p.scale, co[i], si[i]);
  float* out = p.table + row * p.rope_dim + 4 * q;
  *reinterpret_cast<float4*>(out) = make_float4(co[0], co[1], co[2], co[3]);
  *reinterpret_cast<float4*>(out + half) = make_float4(si[0], si[1], si[2], si[3]);
}

}  // namespace loop

cudaError_t launch_rope(const dsv4_rope_params& p, cudaStream_t s) {
  const bool in_place = p.x == p.y && (!p.x2 || p.x2 == p.y2);
  const int pairs = p.rope_halves ? p.rope_dim / 16 : p.rope_dim / 8;
  const int items = pairs + (in_place ? 0 : (p.head_dim - p.rope_dim) / 8);
  const int heads = p.heads + (p.x2 ? p.heads2 : 0);
  int at_once = 256 / items;
  if (at_once > heads) at_once = heads;
  int tokens = 256 / (items * at_once);
  if (tokens > 64) tokens = 64;
  if (tokens > p.T) tokens = p.T;
  const dim3 block(items, at_once, tokens), grid((unsigned)((p.T + (int64_t)tokens - 1) / tokens));
  if (p.dtype == DSV4_F32)
    return p.rope_halves ? launch_pdl(loop::rope_kernel<true, true>, grid, block, 0, s, true, p, pairs)
                         : launch_pdl(loop::rope_kernel<true, false>, grid, block, 0, s, true, p, pairs);
  return p.rope_halves ? launch_pdl(loop::rope_kernel<false, true>, grid, block, 0, s, true, p, pairs)
                       : launch_pdl(loop::rope_kernel<false, false>, grid, block, 0, s, true, p, pairs);
}

cudaError_t launch_rope_table(const dsv4_rope_table_params& p, cudaStream_t s) {
  const int64_t threads = (int64_t)p.rows * (p.rope_dim / 8);
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(loop::rope_table_kernel, dim3((unsigned)blocks), dim3(256), 0, s, true, p);
}

}  // namespace dsv4
