// C ABI entry points of the operators that surround the layers: host-side validation, then the launches.
// Argument meanings and error behaviour are documented in include/dsv4_loop.h.
#include <cmath>
#include <cstdint>

#include "loop_common.cuh"

using namespace dsv4;

namespace {

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
bool act_dtype(int d) { return d == DSV4_F32 || d == DSV4_BF16; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DSV4_OK;
  record_cuda_error((int)e);
  return DSV4_ERR_CUDA;
}

#define CHECK(cond, code) \
  do {                    \
    if (!(cond)) return (code); \
  } while (0)

// Rows of a dsv4_rope call: `heads` of each of T tokens, `row` bytes each (strides in bytes).
struct Rows {
  uintptr_t at;
  int64_t token, head;
  int T, heads;
};

// Whether rows of a and b share memory, for rows whose extents are apart, that begin at one place, or that have their strides
// in common (parts of one buffer); rows of other buffers that are laid through one another are not looked into.
bool rows_meet(Rows a, Rows b, int64_t row) {
  const auto extent = [&](const Rows& r) { return (__int128)(r.T - 1) * r.token + (__int128)(r.heads - 1) * r.head + row; };
  if (a.at + extent(a) <= b.at || b.at + extent(b) <= a.at) return false;
  if (a.at == b.at) return true;
  if (a.T == 1) a.token = b.token = INT64_MAX;
  if (a.heads == 1) a.head = b.head;
  if (b.heads == 1) b.head = a.head;
  if (a.token != b.token || a.head != b.head || a.token <= 0) return false;
  // the wider stride outside; b's rows against a's that lie j narrow strides on from the place where they would meet
  const bool tokens_outside = a.token >= a.head;
  const int64_t wide = tokens_outside ? a.token : a.head, narrow = tokens_outside ? a.head : a.token;
  const int wide_a = tokens_outside ? a.T : a.heads, wide_b = tokens_outside ? b.T : b.heads;
  const int narrow_a = tokens_outside ? a.heads : a.T, narrow_b = tokens_outside ? b.heads : b.T;
  const int64_t off = (int64_t)(b.at - a.at), first = off / wide - (off % wide < 0);
  for (int64_t k = first; k <= first + 1; ++k) {
    if (k >= wide_a || -k >= wide_b) continue;
    const int64_t rest = off - k * wide;  // between -wide and wide
    if (narrow_a == 1 && narrow_b == 1) {
      if (rest < row && -rest < row) return true;
      continue;
    }
    if (narrow <= 0) return rest < row && -rest < row;
    const int64_t j0 = rest / narrow - (rest % narrow < 0);
    for (int64_t j = j0; j <= j0 + 1; ++j)
      if (j < narrow_a && -j < narrow_b && rest - j * narrow < row && j * narrow - rest < row) return true;
  }
  return false;
}

// Whether rows of `dim` elements at t token + h head (strides of dim or more) lie apart from one another.
bool rows_apart(int64_t token, int64_t head, int T, int heads, int dim) {
  if (T <= 1 || heads == 1 || token / heads >= head || head / T >= token) return true;  // one stride holds all of the other's rows
  for (int h = 1; h < heads; ++h) {
    const __int128 at = (__int128)h * head;
    const int64_t rest = (int64_t)(at % token);
    const __int128 t = at / token;
    if ((rest < dim && t < T) || (token - rest < dim && t + 1 < T)) return false;
  }
  return true;
}

// One tensor of a dsv4_rope call.
int check_rope_rows(const void* x, const void* y, int heads, int T, const int64_t (&stride)[4], int head_dim) {
  CHECK(heads >= 1 && heads <= 1024, DSV4_ERR_INVALID);
  for (int64_t s : stride) CHECK(s >= 0 && s % 8 == 0, DSV4_ERR_INVALID);
  CHECK((stride[2] >= head_dim || T <= 1) && (stride[3] >= head_dim || heads == 1), DSV4_ERR_INVALID);
  CHECK(rows_apart(stride[2], stride[3], T, heads, head_dim), DSV4_ERR_INVALID);
  if (T == 0) return DSV4_OK;
  CHECK(x && y && aligned(x, 16) && aligned(y, 16), DSV4_ERR_INVALID);
  CHECK(x != y || (stride[0] == stride[2] && stride[1] == stride[3]), DSV4_ERR_INVALID);
  return DSV4_OK;
}

}  // namespace

extern "C" {

int dsv4_rope_freqs(const dsv4_rope_freqs_params* p, uint64_t* freqs) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_rope_freqs_params) && freqs != nullptr, DSV4_ERR_INVALID);
  const int dim = p->rope_dim, kind = p->scaling;
  CHECK(kind >= DSV4_ROPE_NONE && kind <= DSV4_ROPE_BANDS, DSV4_ERR_UNSUPPORTED);
  CHECK(dim >= (kind == DSV4_ROPE_BASE ? 4 : 2) && dim <= 1024 && dim % 2 == 0, DSV4_ERR_INVALID);
  CHECK(std::isfinite(p->theta) && p->theta > 1.0 && std::isfinite(p->factor) && p->factor >= 1.0, DSV4_ERR_INVALID);
  const double two_pi = 6.283185307179586476925;
  double theta = p->theta, low = 0.0, high = 0.0;
  if (kind == DSV4_ROPE_BASE) {
    theta *= std::pow(p->factor, (double)dim / (dim - 2));
    CHECK(std::isfinite(theta), DSV4_ERR_INVALID);
  }
  if (kind == DSV4_ROPE_YARN || kind == DSV4_ROPE_BANDS)
    CHECK(std::isfinite(p->original_len) && p->original_len > 0.0, DSV4_ERR_INVALID);
  if (kind == DSV4_ROPE_YARN) {
    CHECK(std::isfinite(p->beta_fast) && std::isfinite(p->beta_slow) && p->beta_fast > 0.0 && p->beta_slow > 0.0,
          DSV4_ERR_INVALID);
    const auto pair_of = [&](double b) { return dim * std::log(p->original_len / (b * two_pi)) / (2.0 * std::log(theta)); };
    low = std::fmax(std::floor(pair_of(p->beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(p->beta_slow)), dim - 1.0);
  }
  if (kind == DSV4_ROPE_BANDS)
    CHECK(std::isfinite(p->low_turns) && std::isfinite(p->high_turns) && p->high_turns > p->low_turns, DSV4_ERR_INVALID);
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / dim);
    if (kind == DSV4_ROPE_LINEAR) f /= p->factor;
    if (kind == DSV4_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = f / p->factor * r + f * (1.0 - r);
    }
    if (kind == DSV4_ROPE_BANDS) {
      const double m = (p->original_len * f / two_pi - p->low_turns) / (p->high_turns - p->low_turns);
      const double mix = std::fmin(std::fmax(m, 0.0), 1.0);
      f = (1.0 - mix) * f / p->factor + mix * f;
    }
    freqs[i] = (uint64_t)std::ldexp(f / two_pi, 64);  // (f <= 1: below 2^62)
  }
  return DSV4_OK;
}

int dsv4_rope(const dsv4_rope_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_rope_params), DSV4_ERR_INVALID);
  CHECK(act_dtype(p->dtype), DSV4_ERR_UNSUPPORTED);
  CHECK(p->T >= 0 && p->T <= (1 << 30) && p->head_dim >= 16 && p->head_dim <= 1024 && p->head_dim % 8 == 0,
        DSV4_ERR_INVALID);
  CHECK(p->rope_first >= 0 && p->rope_first % 8 == 0 && p->rope_dim >= 16 && p->rope_dim % 16 == 0 &&
            p->rope_dim <= p->head_dim && p->rope_first <= p->head_dim - p->rope_dim,
        DSV4_ERR_INVALID);
  CHECK((p->rope_halves == 0 || p->rope_halves == 1) && (p->inverse == 0 || p->inverse == 1), DSV4_ERR_INVALID);
  CHECK(std::isfinite(p->scale), DSV4_ERR_INVALID);
  int st = check_rope_rows(p->x, p->y, p->heads, p->T,
                           {p->x_token_stride, p->x_head_stride, p->y_token_stride, p->y_head_stride}, p->head_dim);
  CHECK(st == DSV4_OK, st);
  if (p->x2 != nullptr || p->y2 != nullptr) {
    st = check_rope_rows(p->x2, p->y2, p->heads2, p->T,
                         {p->x2_token_stride, p->x2_head_stride, p->y2_token_stride, p->y2_head_stride}, p->head_dim);
    CHECK(st == DSV4_OK, st);
  }
  if (p->T == 0) return DSV4_OK;
  const int64_t size = p->dtype == DSV4_F32 ? 4 : 2, row = p->head_dim * size;
  const auto rows = [&](const void* at, int64_t token, int64_t head, int heads) {
    return Rows{reinterpret_cast<uintptr_t>(at), token * size, head * size, p->T, heads};
  };
  const Rows x = rows(p->x, p->x_token_stride, p->x_head_stride, p->heads), y = rows(p->y, p->y_token_stride, p->y_head_stride, p->heads);
  CHECK(p->x == p->y || !rows_meet(y, x, row), DSV4_ERR_INVALID);
  if (p->x2 != nullptr) {
    const Rows x2 = rows(p->x2, p->x2_token_stride, p->x2_head_stride, p->heads2);
    const Rows y2 = rows(p->y2, p->y2_token_stride, p->y2_head_stride, p->heads2);
    CHECK(p->x2 == p->y2 || !rows_meet(y2, x2, row), DSV4_ERR_INVALID);
    CHECK(!rows_meet(y, x2, row) && !rows_meet(y2, x, row) && !rows_meet(y, y2, row), DSV4_ERR_INVALID);
  }
  CHECK(p->positions && p->freqs && aligned(p->positions, 4) && aligned(p->freqs, 16), DSV4_ERR_INVALID);
  return cuda_status(launch_rope(*p, (cudaStream_t)stream));
}

int dsv4_rope_table(const dsv4_rope_table_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_rope_table_params), DSV4_ERR_INVALID);
  CHECK(p->rope_dim >= 8 && p->rope_dim <= 1024 && p->rope_dim % 8 == 0, DSV4_ERR_INVALID);
  CHECK(p->rows >= 0 && p->first_position >= 0 && (int64_t)p->first_position + p->rows <= 0x7FFFFFFF &&
            std::isfinite(p->scale),
        DSV4_ERR_INVALID);
  if (p->rows == 0) return DSV4_OK;
  CHECK(p->table && p->freqs && aligned(p->table, 16) && aligned(p->freqs, 16), DSV4_ERR_INVALID);
  return cuda_status(launch_rope_table(*p, (cudaStream_t)stream));
}

int dsv4_batch_plan(const dsv4_batch_plan_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_batch_plan_params), DSV4_ERR_INVALID);
  CHECK(p->B >= 0 && p->B <= DSV4_PLAN_MAX_REQUESTS && p->T >= 0 && p->T <= DSV4_PLAN_MAX_TOKENS, DSV4_ERR_INVALID);
  CHECK(p->num_caches >= 1 && p->num_caches <= DSV4_PLAN_MAX_CACHES, DSV4_ERR_INVALID);
  CHECK(p->q_start && aligned(p->q_start, 4) && aligned(p->positions, 16) && aligned(p->token_seq, 16), DSV4_ERR_INVALID);
  if (p->B > 0)
    CHECK(p->ctx && p->n_new && p->kv_len && aligned(p->ctx, 4) && aligned(p->ctx_add, 4) && aligned(p->n_new, 4) &&
              aligned(p->ctx_out, 4) && aligned(p->kv_len, 4),
          DSV4_ERR_INVALID);
  for (int g = 0; g < p->num_caches; ++g) {
    const dsv4_plan_cache& c = p->caches[g];
    CHECK(c.page_size >= 1 && c.page_size <= 65536 && c.ratio >= 1 && c.ratio <= 65536, DSV4_ERR_INVALID);
    CHECK(c.window >= 0 && (c.window == 0 || c.ratio == 1), DSV4_ERR_INVALID);
    CHECK(c.max_pages_per_seq >= 1 && c.max_pages_per_seq <= (1 << 19), DSV4_ERR_INVALID);
    CHECK(c.num_pages >= 0 && c.num_pages <= 0x7FFFFFFF, DSV4_ERR_INVALID);
    CHECK(c.free_count && c.free_count_out && aligned(c.free_count, 4) && aligned(c.free_count_out, 4), DSV4_ERR_INVALID);
    CHECK(c.num_pages == 0 || (c.free_pages && aligned(c.free_pages, 4)), DSV4_ERR_INVALID);
    CHECK(aligned(c.slots, 16), DSV4_ERR_INVALID);
    CHECK((c.window > 0) == (c.first != nullptr) && (c.window > 0) == (c.first_out != nullptr), DSV4_ERR_INVALID);
    if (p->B > 0)
      CHECK(c.block_table && c.held && c.held_out && aligned(c.block_table, 4) && aligned(c.held, 4) &&
                aligned(c.held_out, 4) && aligned(c.first, 4) && aligned(c.first_out, 4),
            DSV4_ERR_INVALID);
    for (int h = 0; h < g; ++h) {  // what a cache writes is its own
      const dsv4_plan_cache& o = p->caches[h];
      CHECK(c.free_count_out != o.free_count_out && (c.num_pages == 0 || c.free_pages != o.free_pages) &&
                (c.slots == nullptr || c.slots != o.slots) && (p->B == 0 || (c.block_table != o.block_table && c.held_out != o.held_out)) &&
                (c.first_out == nullptr || c.first_out != o.first_out),
            DSV4_ERR_INVALID);
      // ... and is not read for another: a request's numbers of all caches are read and written by one thread in turn
      CHECK(c.free_count_out != o.free_count && o.free_count_out != c.free_count &&
                (p->B == 0 || (c.held_out != o.held && o.held_out != c.held)) &&
                (c.first == nullptr || c.first != o.first_out) && (o.first == nullptr || o.first != c.first_out),
            DSV4_ERR_INVALID);
    }
  }
  return cuda_status(launch_batch_plan(*p, (cudaStream_t)stream));
}

int dsv4_draft_verify(const dsv4_draft_verify_params* p, dsv4_stream_t stream) {
  CHECK(p != nullptr && p->struct_size == sizeof(dsv4_draft_verify_params), DSV4_ERR_INVALID);
  CHECK(p->T >= 0 && p->T <= (1 << 30) && p->B >= 0 && p->B <= 65535 && p->max_q_len >= 1, DSV4_ERR_INVALID);
  CHECK(p->vocab >= 1 && p->vocab <= (1 << 24), DSV4_ERR_INVALID);
  CHECK(act_dtype(p->target_dtype) && (p->draft == nullptr || act_dtype(p->draft_dtype)), DSV4_ERR_UNSUPPORTED);
  CHECK((p->target_probs == 0 || p->target_probs == 1) && (p->draft_probs == 0 || p->draft_probs == 1), DSV4_ERR_INVALID);
  if (p->B == 0) return DSV4_OK;
  CHECK(p->q_start && p->n_out && p->out_tokens && aligned(p->q_start, 4) && aligned(p->n_out, 4) &&
            aligned(p->out_tokens, 4) && aligned(p->logp, 4),
        DSV4_ERR_INVALID);
  if (p->T > 0) {
    CHECK(p->target && p->tokens && aligned(p->target, p->target_dtype == DSV4_F32 ? 4 : 2) && aligned(p->tokens, 4),
          DSV4_ERR_INVALID);
    CHECK(p->target_stride >= p->vocab, DSV4_ERR_INVALID);
    CHECK((p->u == nullptr) == (p->noise == nullptr), DSV4_ERR_INVALID);
  }
  CHECK(aligned(p->temperature, 4) && aligned(p->u, 4) && aligned(p->noise, 4) && aligned(p->draft_row, 4), DSV4_ERR_INVALID);
  CHECK(p->noise == nullptr || p->noise_stride >= p->vocab, DSV4_ERR_INVALID);
  if (p->draft != nullptr) {
    CHECK(aligned(p->draft, p->draft_dtype == DSV4_F32 ? 4 : 2) && p->draft_stride >= p->vocab && p->draft_rows >= 0,
          DSV4_ERR_INVALID);
  }
  return cuda_status(launch_draft_verify(*p, (cudaStream_t)stream));
}

}  // extern "C"
