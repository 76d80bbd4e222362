// Which kernel a grouped-query attention call runs.
#include "gqa_attention.cuh"

namespace dsv4 {

// Up to 32 rows of (token, head) for each kv head of a sequence: the streaming kernel, whose cost is the
// cache's bytes; more: the tcgen05 kernel, which fills 128 rows of an MMA.  (32 x 8k e4m3 rows, 8 rows a kv head: 63 us,
// 278 on the tcgen05 kernel; one token over 777 rows 8.0 and 20.9; at 32 rows, 48 x 4000 rows of 4 kv heads, e4m3 96 and
// 155, bf16 70 and 76, capped bf16 in a window of 1024 36 and 62.)  The bound of the call decides, so one long chunk takes
// every sequence beside it along (512 tokens beside 31 single ones over up to 8k e4m3 rows: 337 us, as two calls 151;
// bf16 177 and 182).
static bool use_decode(const dsv4_gqa_attention_params& p) {
  const int64_t max_n = p.max_q_len < p.T ? p.max_q_len : p.T;
  return max_n * (p.q_heads / p.kv_heads) <= 32;
}

size_t gqa_attention_workspace(const dsv4_gqa_attention_params& p) {
  if (p.T == 0 || p.B == 0) return 256;
  return use_decode(p) ? gqa::decode_workspace(p) : gqa::prefill_workspace(p);
}

cudaError_t launch_gqa_attention(const dsv4_gqa_attention_params& p, cudaStream_t s) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  return use_decode(p) ? gqa::launch_decode(p, s) : gqa::launch_prefill(p, s);
}

}  // namespace dsv4
