// Shared pieces of the grouped-query kernels: the ragged batch and the paged per-head caches.
#pragma once

#include "../../include/dsv4_gqa.h"
#include "dsv4_common.cuh"
#include "dsv4_launch.h"

namespace dsv4 {

cudaError_t launch_gqa_append(const dsv4_gqa_append_params& p, cudaStream_t s);
cudaError_t read_flags_gqa_append(uint32_t* f);
size_t gqa_attention_workspace(const dsv4_gqa_attention_params& p);
cudaError_t launch_gqa_attention(const dsv4_gqa_attention_params& p, cudaStream_t s);
cudaError_t read_flags_gqa_decode(uint32_t* f);
cudaError_t read_flags_gqa_prefill(uint32_t* f);

namespace gqa {

struct Seq {
  int t0, n, kv;  // first flat token, new tokens, rows including them
  bool ok;        // false: the sequence is skipped
};

constexpr int MAX_ROWS = 1 << 30;  // of a sequence

// Sequence b of the batch.
__device__ __forceinline__ Seq sequence(const int32_t* q_start, const int32_t* kv_len, int b, int T, int max_q_len,
                                        int kv_bound) {
  Seq s;
  s.t0 = q_start[b];
  const int t1 = q_start[b + 1];
  s.kv = kv_len[b];
  s.ok = s.t0 >= 0 && t1 >= s.t0 && t1 <= T;
  s.n = s.ok ? t1 - s.t0 : 0;
  s.ok = s.ok && s.n <= max_q_len && s.kv >= s.n && s.kv <= min(kv_bound, MAX_ROWS);
  return s;
}

}  // namespace gqa
}  // namespace dsv4
