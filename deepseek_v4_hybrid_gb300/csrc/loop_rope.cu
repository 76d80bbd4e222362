// Rotary positions: rows turned by their tokens' positions, and the cos / sin tables.
//
// An angle is position * f_i / (2 pi) turns.  With the frequency as a 64-bit binary fraction of a turn, the product
// modulo 2^64 is the angle reduced to one turn, exactly, for every position: one integer product in the place of
// a reduction by 2 pi in wider floating point.  Its 64 bits are split into the nearest quarter turn and a rest that
// becomes an fp32 number of half turns, so that a sine or cosine near 0 keeps its relative accuracy.
//
// A thread owns 16 bytes (with halves, and the 16 of their partners) of a token's heads and turns that chunk of head after
// head; the block computes each token's angles once, while the first chunks are on their way.
// Bound by HBM: 16384 tokens of 72 heads of 128 bf16 (604 MB) 88 us, 6.8 TB/s; 4096 of 32 heads of 128 fp32 (134 MB) 22 us; 9377
// of 24 heads of 64, half turned (58 MB), 13 us; 48 tokens 2.8 us from a graph, a launch (called one by one from
// Python 3.4, the host's time); a table of 131072 rows of 64 (34 MB) 8.6 us.
#include "loop_common.cuh"

namespace dsv4 {
namespace loop {

// cos and sin of position p under a frequency, times scale.  Within an eighth of a turn the Taylor sums of sin and cos
// up to the 9th and 10th power are off by less than 2^-28 and 2^-32 of them.
__device__ __forceinline__ void turn(uint32_t p, uint64_t freq, float scale, float& co, float& si) {
  constexpr double PI = 3.14159265358979323846, P2 = PI * PI;
  constexpr float S0 = (float)PI, S0_LOW = (float)(PI - (double)(float)PI), S1 = (float)(-P2 * PI / 6),
                  S2 = (float)(P2 * P2 * PI / 120), S3 = (float)(-P2 * P2 * P2 * PI / 5040),
                  S4 = (float)(P2 * P2 * P2 * P2 * PI / 362880);
  constexpr float C1 = (float)(-P2 / 2), C2 = (float)(P2 * P2 / 24), C3 = (float)(-P2 * P2 * P2 / 720),
                  C4 = (float)(P2 * P2 * P2 * P2 / 40320), C5 = (float)(-P2 * P2 * P2 * P2 * P2 / 3628800);
  const uint64_t t = p * freq, quadrant = (t + (1ull << 61)) >> 62;
  const float h = __ll2float_rn((long long)(t - (quadrant << 62))) * 0x1p-63f, z = h * h;  // half turns, |h| <= 1/4
  const float s = fmaf(h, S0, h * fmaf(z, fmaf(z, fmaf(z, fmaf(z, S4, S3), S2), S1), S0_LOW));
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, C5, C4), C3), C2), C1), 1.f);
  const float a = quadrant & 1 ? s : c, b = quadrant & 1 ? c : s;
  co = (quadrant + 1) & 2 ? -scale * a : scale * a;
  si = quadrant & 2 ? -scale * b : scale * b;
}

// 16 bytes of a row: E elements.
template <bool F32>
struct Chunk {
  static constexpr int E = F32 ? 4 : 8;
  uint4 w;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + at * (16 / E));
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(base) + at * (16 / E)) = w;
  }
  __device__ __forceinline__ void get(float (&v)[E]) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < E; ++i)
      v[i] = __uint_as_float(F32 ? x[i % 4] : i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[E]) {
    if (F32)
      w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      w = make_uint4(float2_to_bf16x2_bits(v[0], v[1]), float2_to_bf16x2_bits(v[2], v[3]),
                     float2_to_bf16x2_bits(v[4 % E], v[5 % E]), float2_to_bf16x2_bits(v[6 % E], v[7 % E]));
  }
};

// blockDim = (items of a head, heads at once, tokens).  Item c < pairs turns a chunk (halves: and its partner), the
// others copy one.  A thread loads N chunks of different heads side by side, the first ones before the angles are known;
// the block computes each token's angles once.
template <bool F32, bool HALVES, int N>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ dsv4_rope_params p, int pairs) {
  constexpr int E = Chunk<F32>::E, NP = HALVES ? E : E / 2, NC = HALVES ? 2 : 1;  // pairs, and chunks, of an item
  extern __shared__ float2 table[];  // cos and sin of [tokens, rope_dim / 2]
  pdl_wait();
  pdl_launch_dependents();
  const int c = threadIdx.x, half = p.rope_dim / 2, step = blockDim.y;
  const int64_t t0 = (int64_t)blockIdx.x * blockDim.z, t = t0 + threadIdx.z;
  const bool here = t < p.T, turned = c < pairs;
  int d = p.rope_first + E * c;  // first dim of the chunk
  if (!turned) {
    d = E * (c - pairs);
    if (d >= p.rope_first) d += p.rope_dim;
  }
  const int all = here ? p.heads + (p.x2 ? p.heads2 : 0) : 0;
  Chunk<F32> u[N][NC];
  const auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * step;
      if (h >= all) continue;
      const bool second = h >= p.heads;
      const void* x = second ? p.x2 : p.x;
      const int64_t from = second ? t * p.x2_token_stride + (h - p.heads) * p.x2_head_stride + d
                                  : t * p.x_token_stride + h * p.x_head_stride + d;
      u[i][0].load(x, from);
      if (HALVES && turned) u[i][NC - 1].load(x, from + half);
    }
  };
  load(threadIdx.y);
  const int pos = here ? p.positions[t] : -1;
  const int threads = blockDim.x * blockDim.y * blockDim.z;
  for (int i = threadIdx.x + blockDim.x * (threadIdx.y + step * threadIdx.z); i < (int)blockDim.z * half; i += threads) {
    const int z = blockDim.z == 1 ? 0 : i / half;
    if (t0 + z >= p.T) break;
    float2 cs;
    turn((uint32_t)p.positions[t0 + z], p.freqs[i - z * half], p.scale, cs.x, cs.y);
    if (p.inverse) cs.y = -cs.y;
    table[i] = cs;
  }
  __syncthreads();
  if (pos < 0) return;
  float co[NP], si[NP];
  if (turned) {
    const float4* cs = reinterpret_cast<const float4*>(table + threadIdx.z * half + NP * c);
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
      const float4 a = cs[i / 2];
      co[i] = a.x, si[i] = a.y, co[i + 1] = a.z, si[i + 1] = a.w;
    }
  }
  for (int h0 = threadIdx.y; h0 < all; h0 += N * step) {
    if (h0 != threadIdx.y) load(h0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * step;
      if (h >= all) continue;
      const bool second = h >= p.heads;
      void* y = second ? p.y2 : p.y;
      const int64_t to = second ? t * p.y2_token_stride + (h - p.heads) * p.y2_head_stride + d
                                : t * p.y_token_stride + h * p.y_head_stride + d;
      if (turned) {
        float a[E], b[E];
        u[i][0].get(a);
        if (HALVES) {
          u[i][NC - 1].get(b);
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const float a0 = a[j], b0 = b[j];
            a[j] = a0 * co[j % NP] - b0 * si[j % NP];
            b[j] = b0 * co[j % NP] + a0 * si[j % NP];
          }
          u[i][NC - 1].set(b);
          u[i][NC - 1].store(y, to + half);
        } else {
#pragma unroll
          for (int j = 0; j < E / 2; ++j) {
            const float a0 = a[2 * j], b0 = a[2 * j + 1];
            a[2 * j] = a0 * co[j] - b0 * si[j];
            a[2 * j + 1] = b0 * co[j] + a0 * si[j];
          }
        }
        u[i][0].set(a);
      }
      u[i][0].store(y, to);
    }
  }
}

// Four pairs of a row a thread; blockDim = (rope_dim / 8, rows).
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ dsv4_rope_table_params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;
  const ulonglong2* f = reinterpret_cast<const ulonglong2*>(p.freqs) + 2 * threadIdx.x;
  const ulonglong2 f0 = f[0], f1 = f[1];
  const uint64_t freq[4] = {f0.x, f0.y, f1.x, f1.y};
  float co[4], si[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) turn((uint32_t)(p.first_position + row), freq[i], p.scale, co[i], si[i]);
  float* out = p.table + row * p.rope_dim + 4 * threadIdx.x;
  *reinterpret_cast<float4*>(out) = make_float4(co[0], co[1], co[2], co[3]);
  *reinterpret_cast<float4*>(out + p.rope_dim / 2) = make_float4(si[0], si[1], si[2], si[3]);
}

}  // namespace loop

cudaError_t launch_rope(const dsv4_rope_params& p, cudaStream_t s) {
  const bool in_place = p.x == p.y && (!p.x2 || p.x2 == p.y2);
  const int unit = p.dtype == DSV4_F32 ? 4 : 8;
  const int pairs = p.rope_halves ? p.rope_dim / (2 * unit) : p.rope_dim / unit;
  const int items = pairs + (in_place ? 0 : (p.head_dim - p.rope_dim) / unit);
  // Six vectors of a thread are on their way at once (four: 16384 tokens of 72 heads 101 us for 88; with partners, eight: 9377
  // tokens of 24 heads of 64 14.5 us for 12.5).
  const int N = p.rope_halves ? 3 : 6;
  const int heads = p.heads + (p.x2 ? p.heads2 : 0), enough = (heads + N - 1) / N;
  int at_once = 256 / items;
  if (at_once > enough) at_once = enough;
  int tokens = 256 / (items * at_once);
  if (tokens > 64) tokens = 64;
  if (tokens > p.T) tokens = p.T;
  const size_t smem = (size_t)tokens * (p.rope_dim / 2) * sizeof(float2);
  const dim3 block(items, at_once, tokens), grid((unsigned)((p.T + (int64_t)tokens - 1) / tokens));
  if (p.dtype == DSV4_F32)
    return p.rope_halves ? launch_pdl(loop::rope_kernel<true, true, 3>, grid, block, smem, s, true, p, pairs)
                         : launch_pdl(loop::rope_kernel<true, false, 6>, grid, block, smem, s, true, p, pairs);
  return p.rope_halves ? launch_pdl(loop::rope_kernel<false, true, 3>, grid, block, smem, s, true, p, pairs)
                       : launch_pdl(loop::rope_kernel<false, false, 6>, grid, block, smem, s, true, p, pairs);
}

cudaError_t launch_rope_table(const dsv4_rope_table_params& p, cudaStream_t s) {
  const int quads = p.rope_dim / 8, rows = 256 / quads;
  return launch_pdl(loop::rope_table_kernel, dim3((unsigned)((p.rows + (int64_t)rows - 1) / rows)), dim3(quads, rows), 0, s,
                    true, p);
}

}  // namespace dsv4
