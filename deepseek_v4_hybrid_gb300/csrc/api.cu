// C ABI entry points: host-side argument validation, then the kernel launches.
// The declarations, argument meanings and error behaviour are documented in include/dsv4.h.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "dsv4_common.cuh"
#include "dsv4_launch.h"
#include "gqa_common.cuh"

using namespace dsv4;

namespace {

thread_local int g_last_cuda_error = 0;
std::atomic<unsigned long long> g_kernel_launches{0};

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DSV4_OK;
  g_last_cuda_error = (int)e;
  return DSV4_ERR_CUDA;
}

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

bool latent_cache_dtype(int d) { return d == DSV4_F32 || d == DSV4_BF16 || d == DSV4_FP8_DS_MLA; }
bool act_dtype(int d) { return d == DSV4_F32 || d == DSV4_BF16; }

#define CHECK(cond, code) \
  do {                    \
    if (!(cond)) return (code); \
  } while (0)

// What the two grouped-query calls share: the ragged batch, the caches and their exponents.
template <typename P>
int check_gqa(const P& p) {
  CHECK(p.T >= 0 && p.T <= (1 << 30) && p.B >= 0 && p.B <= 65535 && p.max_q_len >= 1, DSV4_ERR_INVALID);
  CHECK(p.num_pages >= 0 && p.num_pages <= 0x7FFFFFFF && p.max_pages_per_seq > 0, DSV4_ERR_INVALID);
  CHECK(p.q_heads >= 1 && p.q_heads <= 1024 && p.kv_heads >= 1 && p.kv_heads <= 1024, DSV4_ERR_INVALID);
  CHECK(p.head_dim == 64 || p.head_dim == 128, DSV4_ERR_UNSUPPORTED);
  CHECK(p.page_size == 16 || p.page_size == 32 || p.page_size == 64 || p.page_size == 128 || p.page_size == 256,
        DSV4_ERR_UNSUPPORTED);
  CHECK(p.cache_dtype == DSV4_BF16 || p.cache_dtype == DSV4_E4M3_PAGE, DSV4_ERR_UNSUPPORTED);
  if (p.T == 0 || p.B == 0) return DSV4_OK;
  CHECK(p.k_cache && p.v_cache && p.block_table && p.q_start && p.kv_len, DSV4_ERR_INVALID);
  CHECK(aligned(p.k_cache, 16) && aligned(p.v_cache, 16) && aligned(p.block_table, 4) && aligned(p.q_start, 4) &&
            aligned(p.kv_len, 4),
        DSV4_ERR_INVALID);
  const int64_t unit = p.cache_dtype == DSV4_BF16 ? 8 : 16;  // elements of 16 bytes
  const int64_t strides[] = {p.k_page_stride, p.k_cache_head_stride, p.k_row_stride,
                             p.v_page_stride, p.v_cache_head_stride, p.v_row_stride};
  for (int64_t x : strides) CHECK(x > 0 && x % unit == 0, DSV4_ERR_INVALID);
  CHECK(p.k_row_stride >= p.head_dim && p.v_row_stride >= p.head_dim, DSV4_ERR_INVALID);
  CHECK(p.cache_dtype == DSV4_BF16 || (p.k_exp && p.v_exp), DSV4_ERR_INVALID);
  return DSV4_OK;
}

bool token_strides(int64_t token, int64_t head) { return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0; }

}  // namespace

void dsv4::record_cuda_error(int e) { g_last_cuda_error = e; }

cudaError_t dsv4::count_launch(cudaError_t e) {
  if (e == cudaSuccess) g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

extern "C" {

int dsv4_abi_version(void) { return DSV4_ABI_VERSION; }

uint64_t dsv4_kernel_launches(void) { return g_kernel_launches.load(std::memory_order_relaxed); }

const char* dsv4_status_string(int s) {
  switch (s) {
    case DSV4_OK: return "ok";
    case DSV4_ERR_INVALID: return "invalid argument";
    case DSV4_ERR_UNSUPPORTED: return "unsupported dtype or shape";
    case DSV4_ERR_CUDA: return "CUDA error";
    case DSV4_ERR_BOUNDS: return "a kernel skipped an out-of-range index";
    case DSV4_ERR_TIMEOUT: return "a kernel gave up a bounded wait (outputs unspecified)";
  }
  return "unknown status";
}

int dsv4_last_cuda_error(void) { return g_last_cuda_error; }

int dsv4_read_device_flags(uint32_t* flags) {
  CHECK(flags != nullptr, DSV4_ERR_INVALID);
  *flags = 0;
  int st = cuda_status(cudaDeviceSynchronize());
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_insert_compress(flags));
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_indexer(flags));
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_attention(flags));
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_gqa_append(flags));
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_gqa_prefill(flags));
  if (st != DSV4_OK) return st;
  st = cuda_status(read_flags_gqa_decode(flags));
  if (st != DSV4_OK) return st;
  if (*flags & 4u) return DSV4_ERR_TIMEOUT;
  return *flags ? DSV4_ERR_BOUNDS : DSV4_OK;
}

int dsv4_kv_insert(const dsv4_kv_insert_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_kv_insert_params), DSV4_ERR_INVALID);
  CHECK(p->T >= 0 && p->page_size > 0 && p->num_pages >= 0, DSV4_ERR_INVALID);
  CHECK(act_dtype(p->kv_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(latent_cache_dtype(p->cache_dtype), DSV4_ERR_UNSUPPORTED);
  if (p->T == 0) return DSV4_OK;
  CHECK(p->kv_new && p->slot_mapping && p->cache, DSV4_ERR_INVALID);
  CHECK(aligned(p->kv_new, 8) && aligned(p->cache, 16) && aligned(p->slot_mapping, 8), DSV4_ERR_INVALID);
  CHECK(p->cos_sin == nullptr || (p->positions != nullptr && p->max_pos > 0), DSV4_ERR_INVALID);
  return cuda_status(launch_kv_insert(*p, (cudaStream_t)stream));
}

int dsv4_qnorm_rope_kv_insert(const dsv4_qnorm_rope_kv_insert_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_qnorm_rope_kv_insert_params), DSV4_ERR_INVALID);
  CHECK(p->T >= 0 && p->page_size > 0 && p->num_pages >= 0, DSV4_ERR_INVALID);
  CHECK(p->H >= 1 && p->H_pad >= p->H && p->H_pad <= 1024, DSV4_ERR_INVALID);
  CHECK(act_dtype(p->act_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(latent_cache_dtype(p->cache_dtype), DSV4_ERR_UNSUPPORTED);
  if (p->T == 0) return DSV4_OK;
  CHECK(p->q && p->q_out && p->kv_new && p->slot_mapping && p->cache, DSV4_ERR_INVALID);
  CHECK(aligned(p->q, 16) && aligned(p->q_out, 16) && aligned(p->kv_new, 8) && aligned(p->cache, 16) &&
            aligned(p->slot_mapping, 8) && aligned(p->q_norm_weight, 4),
        DSV4_ERR_INVALID);
  const bool rope = p->apply_q_rope || p->apply_kv_rope;
  CHECK(!rope || (p->positions != nullptr && p->cos_sin != nullptr && p->max_pos > 0), DSV4_ERR_INVALID);
  // q_out is q itself (in place, same head count) or a separate buffer
  const size_t esz = p->act_dtype == DSV4_F32 ? 4 : 2;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(p->q), q1 = q0 + (size_t)p->T * p->H * D * esz;
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(p->q_out), o1 = o0 + (size_t)p->T * p->H_pad * D * esz;
  CHECK((q0 == o0 && p->H_pad == p->H) || o1 <= q0 || q1 <= o0, DSV4_ERR_INVALID);
  return cuda_status(launch_qnorm_rope_kv_insert(*p, (cudaStream_t)stream));
}

int dsv4_padded_num_q_heads(int H, int cache_dtype) {
  if (H < 1 || !latent_cache_dtype(cache_dtype)) return -1;
  return cache_dtype == DSV4_F32 ? H : (H + 63) / 64 * 64;
}

int dsv4_compress_update(const dsv4_compress_update_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_compress_update_params), DSV4_ERR_INVALID);
  CHECK(p->B >= 0 && p->q_per_seq >= 1 && p->q_per_seq <= DSV4_MAX_Q_PER_SEQ, DSV4_ERR_INVALID);
  CHECK((int64_t)p->B * p->q_per_seq == p->T, DSV4_ERR_INVALID);
  CHECK((p->ratio == 4 && p->coff == 2) || (p->ratio == 128 && p->coff == 1) || (p->ratio == 4 && p->coff == 1),
        DSV4_ERR_UNSUPPORTED);
  CHECK(p->q_per_seq <= p->ratio, DSV4_ERR_UNSUPPORTED);
  CHECK(latent_cache_dtype(p->cache_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(p->page_size > 0 && p->num_pages >= 0 && p->max_pages_per_seq > 0 && p->max_pos > 0, DSV4_ERR_INVALID);
  CHECK(p->eps >= 0.f, DSV4_ERR_INVALID);
  if (p->B == 0) return DSV4_OK;
  CHECK(p->kv_score && p->positions && p->state && p->norm_weight && p->cos_sin && p->main_cache && p->block_table,
        DSV4_ERR_INVALID);
  CHECK(aligned(p->kv_score, 8) && aligned(p->state, 8) && aligned(p->norm_weight, 8) &&
            aligned(p->main_cache, 16) && (p->ape == nullptr || aligned(p->ape, 8)),
        DSV4_ERR_INVALID);
  if (p->wk != nullptr) {
    CHECK(p->ik_dim == 64 || p->ik_dim == 128, DSV4_ERR_UNSUPPORTED);
    CHECK(p->ik_dtype == DSV4_F32 || p->ik_dtype == DSV4_BF16 || p->ik_dtype == DSV4_I8_ROWSCALE ||
              p->ik_dtype == DSV4_MXFP4,
          DSV4_ERR_UNSUPPORTED);
    CHECK(p->ik_norm_weight && p->ik_cache && p->ik_block_table && p->ik_max_pages > 0 && p->ik_num_pages >= 0 &&
              p->ik_eps >= 0.f,
          DSV4_ERR_INVALID);
    CHECK(aligned(p->wk, 4) && aligned(p->ik_norm_weight, 4) && aligned(p->ik_cache, 16), DSV4_ERR_INVALID);
  }
  return cuda_status(launch_compress_update(*p, (cudaStream_t)stream));
}

size_t dsv4_indexer_topk_workspace_bytes(const dsv4_indexer_topk_params* p) {
  if (p == nullptr || p->struct_size != sizeof(dsv4_indexer_topk_params) || p->ratio <= 0 || p->T < 0 ||
      p->max_context < 0)
    return 0;
  return indexer_topk_workspace(*p);
}

int dsv4_indexer_topk(const dsv4_indexer_topk_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_indexer_topk_params), DSV4_ERR_INVALID);
  CHECK(p->B >= 0 && p->q_per_seq >= 1 && p->q_per_seq <= DSV4_MAX_Q_PER_SEQ, DSV4_ERR_INVALID);
  CHECK((int64_t)p->B * p->q_per_seq == p->T, DSV4_ERR_INVALID);
  CHECK(p->ratio > 0 && p->page_size > 0 && p->max_pages_per_seq > 0 && p->num_pages >= 0, DSV4_ERR_INVALID);
  CHECK(p->topk > 0 && p->topk <= 16384 && p->max_context >= 0, DSV4_ERR_INVALID);
  CHECK(act_dtype(p->q_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(p->k_dtype == DSV4_F32 || p->k_dtype == DSV4_BF16 || p->k_dtype == DSV4_I8_ROWSCALE ||
            (p->k_dtype == DSV4_MXFP4 && p->head_dim % 32 == 0),
        DSV4_ERR_UNSUPPORTED);
  CHECK(p->n_heads >= 1 && p->n_heads <= 128 && p->head_dim >= 16 && p->head_dim <= 256 && p->head_dim % 16 == 0,
        DSV4_ERR_UNSUPPORTED);
  CHECK((int64_t)p->q_per_seq * p->n_heads <= 256, DSV4_ERR_UNSUPPORTED);
  CHECK(p->max_context / p->ratio <= (1 << 20), DSV4_ERR_UNSUPPORTED);
  if (p->cand_block_size != 0) {
    const int cb = p->cand_block_size;
    CHECK(cb >= 128 && cb <= 65536 && (cb & (cb - 1)) == 0, DSV4_ERR_INVALID);
    CHECK(p->cand_topk >= 1 && p->cand_topk <= 64 && (p->cand_write == 0 || p->cand_write == 1), DSV4_ERR_INVALID);
    CHECK(p->T == 0 || (p->cand_blocks != nullptr && aligned(p->cand_blocks, 4)), DSV4_ERR_INVALID);
  }
  if (p->T == 0) return DSV4_OK;
  CHECK(p->q && p->weights && p->k_cache && p->block_table && p->positions && p->topk_idx, DSV4_ERR_INVALID);
  CHECK(aligned(p->q, 16) && aligned(p->k_cache, 16) && aligned(p->weights, 4), DSV4_ERR_INVALID);
  CHECK(p->workspace != nullptr && aligned(p->workspace, 256), DSV4_ERR_INVALID);
  CHECK(p->workspace_bytes >= indexer_topk_workspace(*p), DSV4_ERR_INVALID);
  return cuda_status(launch_indexer_topk(*p, (cudaStream_t)stream));
}

size_t dsv4_sparse_mla_decode_workspace_bytes(const dsv4_sparse_mla_decode_params* p) {
  if (p == nullptr || p->struct_size != sizeof(dsv4_sparse_mla_decode_params) || p->T < 0 || p->H <= 0 ||
      p->max_context < 0 || p->ratio < 0)
    return 0;
  return sparse_mla_workspace(*p);
}

int dsv4_sparse_mla_decode(const dsv4_sparse_mla_decode_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_sparse_mla_decode_params), DSV4_ERR_INVALID);
  CHECK(p->B >= 0 && p->q_per_seq >= 1 && p->q_per_seq <= DSV4_MAX_Q_PER_SEQ, DSV4_ERR_INVALID);
  CHECK((int64_t)p->B * p->q_per_seq == p->T, DSV4_ERR_INVALID);
  CHECK(p->H >= 1 && p->H <= 128, DSV4_ERR_UNSUPPORTED);
  CHECK(p->page_size > 0 && p->window >= 1 && p->ratio >= 0 && p->max_context >= 0, DSV4_ERR_INVALID);
  CHECK(p->swa_max_pages > 0 && p->swa_num_pages >= 0, DSV4_ERR_INVALID);
  CHECK(act_dtype(p->q_dtype) && act_dtype(p->out_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(latent_cache_dtype(p->cache_dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(p->topk_idx == nullptr || (p->topk > 0 && p->topk <= 16384), DSV4_ERR_INVALID);
  if (p->T == 0) return DSV4_OK;
  CHECK(p->q && p->positions && p->swa_cache && p->swa_block_table && p->out, DSV4_ERR_INVALID);
  if (p->ratio > 0) CHECK(p->main_cache && p->main_block_table && p->main_max_pages > 0, DSV4_ERR_INVALID);
  CHECK(aligned(p->q, 16) && aligned(p->swa_cache, 16) && aligned(p->out, 16), DSV4_ERR_INVALID);
  if (p->ratio > 0) CHECK(aligned(p->main_cache, 16), DSV4_ERR_INVALID);
  CHECK(p->workspace != nullptr && aligned(p->workspace, 256), DSV4_ERR_INVALID);
  CHECK(p->workspace_bytes >= sparse_mla_workspace(*p), DSV4_ERR_INVALID);
  return cuda_status(launch_sparse_mla_decode(*p, (cudaStream_t)stream));
}

int dsv4_gqa_append(const dsv4_gqa_append_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_gqa_append_params), DSV4_ERR_INVALID);
  const int st = check_gqa(*p);
  CHECK(st == DSV4_OK, st);
  if (p->cos_sin != nullptr) {
    CHECK(p->max_pos > 0 && p->rope_first >= 0 && p->rope_first % 8 == 0 && p->rope_dim >= 16 &&
              p->rope_dim % 16 == 0 && p->rope_dim <= p->head_dim && p->rope_first <= p->head_dim - p->rope_dim &&
              aligned(p->cos_sin, 16),
          DSV4_ERR_INVALID);
  }
  if (p->T == 0 || p->B == 0) return DSV4_OK;
  CHECK(p->k_new && p->v_new && aligned(p->k_new, 16) && aligned(p->v_new, 16), DSV4_ERR_INVALID);
  CHECK(token_strides(p->k_token_stride, p->k_head_stride) && token_strides(p->v_token_stride, p->v_head_stride),
        DSV4_ERR_INVALID);
  if (p->q != nullptr) {
    CHECK(p->q_out && aligned(p->q, 16) && aligned(p->q_out, 16), DSV4_ERR_INVALID);
    CHECK(token_strides(p->q_token_stride, p->q_head_stride) &&
              token_strides(p->q_out_token_stride, p->q_out_head_stride),
          DSV4_ERR_INVALID);
    CHECK((p->q_out_token_stride > 0 || p->T == 1) && (p->q_out_head_stride > 0 || p->q_heads == 1), DSV4_ERR_INVALID);
    CHECK(p->q != p->q_out || (p->q_token_stride == p->q_out_token_stride && p->q_head_stride == p->q_out_head_stride),
          DSV4_ERR_INVALID);
  }
  return cuda_status(launch_gqa_append(*p, (cudaStream_t)stream));
}

namespace {
int check_gqa_attention(const dsv4_gqa_attention_params& p) {
  const int st = check_gqa(p);
  CHECK(st == DSV4_OK, st);
  CHECK(p.q_heads % p.kv_heads == 0, DSV4_ERR_INVALID);
  CHECK(p.max_kv_len >= 0 && p.max_kv_len <= (1 << 30) && p.window >= 0, DSV4_ERR_INVALID);
  CHECK((int64_t)(p.max_q_len < p.T ? p.max_q_len : p.T) * (p.q_heads / p.kv_heads) <= (1 << 30), DSV4_ERR_UNSUPPORTED);
  CHECK(p.causal == 0 || p.causal == 1, DSV4_ERR_INVALID);
  CHECK(std::isfinite(p.softmax_scale) && std::isfinite(p.softcap) && p.softcap >= 0.f, DSV4_ERR_INVALID);
  CHECK(std::isfinite(4.f * p.softmax_scale) && p.softcap <= 1024.f, DSV4_ERR_INVALID);
  if (p.softcap > 0.f)
    CHECK(std::isfinite(4.f / p.softcap) && std::isfinite(4.f * p.softmax_scale / p.softcap), DSV4_ERR_INVALID);
  CHECK(act_dtype(p.out_dtype), DSV4_ERR_UNSUPPORTED);
  return DSV4_OK;
}
}  // namespace

size_t dsv4_gqa_attention_workspace_bytes(const dsv4_gqa_attention_params* p) {
  if (p == nullptr || p->struct_size != sizeof(dsv4_gqa_attention_params) || check_gqa_attention(*p) != DSV4_OK)
    return 0;
  return gqa_attention_workspace(*p);
}

int dsv4_gqa_attention(const dsv4_gqa_attention_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_gqa_attention_params), DSV4_ERR_INVALID);
  const int st = check_gqa_attention(*p);
  CHECK(st == DSV4_OK, st);
  if (p->T == 0 || p->B == 0) return DSV4_OK;
  CHECK(p->q && p->out && aligned(p->q, 16) && aligned(p->out, 16) && aligned(p->lse, 4), DSV4_ERR_INVALID);
  CHECK(token_strides(p->q_token_stride, p->q_head_stride), DSV4_ERR_INVALID);
  CHECK(aligned(p->prefix_len, 4) && aligned(p->kv_start, 4) && aligned(p->slopes, 4) && aligned(p->sink, 4),
        DSV4_ERR_INVALID);
  CHECK(p->workspace != nullptr && aligned(p->workspace, 256), DSV4_ERR_INVALID);
  CHECK(p->workspace_bytes >= gqa_attention_workspace(*p), DSV4_ERR_INVALID);
  return cuda_status(launch_gqa_attention(*p, (cudaStream_t)stream));
}

}  // extern "C"
