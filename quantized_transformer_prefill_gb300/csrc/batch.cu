// batch.cu -- C ABI of the batch operators (include/minfer.h): the checks of
// host arguments, then one launcher call.  Nothing here allocates, waits or
// throws, so every entry point can be captured into a CUDA graph.
#include <climits>
#include <cmath>

#include "../../include/minfer.h"
#include "kernels.h"

using namespace minfer;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxHeads = 65535;  // a row of heads is indexed with 32 bits

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool type_ok(int t) { return t == MINFER_F32 || t == MINFER_F16 || t == MINFER_BF16; }
int type_size(int t) { return t == MINFER_F32 ? 4 : 2; }
// a stride of `n` elements between `count` things, which must keep 16-byte alignment if
// there is more than one
bool stride_ok(int64_t n, int64_t count, int t) { return count == 1 || (n >= 0 && (n * type_size(t)) % 16 == 0); }
bool fits31(int64_t a, int64_t b) { return a * b <= INT_MAX; }  // a, b <= INT_MAX each

int from_cuda(cudaError_t e) { return e == cudaSuccess ? MINFER_OK : MINFER_ERR_CUDA; }

// SMs of the current device; 0 without one.  The count of a device never
// changes, so it is asked for once.
int current_sms() {
  static int known[kMaxDevices];  // written with the same value by every thread
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  }
  return n;
}

int check_cache(const minfer_paged_cache* c, PagedCache* out) {
  if (!c || !c->k || !c->v || c->n_pages <= 0 || c->page_size <= 0 || c->n_head_kv <= 0)
    return MINFER_ERR_ARG;
  if (!type_ok(c->type) || (c->head_dim != 64 && c->head_dim != 128)) return MINFER_ERR_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || !stride_ok(c->page_stride, c->n_pages, c->type) ||
      !stride_ok(c->row_stride, c->page_size, c->type) || !stride_ok(c->head_stride, c->n_head_kv, c->type))
    return MINFER_ERR_ARG;
  if (!fits31(c->n_pages, c->page_size)) return MINFER_ERR_TOO_LARGE;
  // (strides between things of which there is one are never used; as 0 they do no harm)
  *out = PagedCache{c->k, c->v, c->n_pages, c->page_size, c->n_head_kv, c->head_dim,
                    c->n_pages > 1 ? c->page_stride : 0, c->page_size > 1 ? c->row_stride : 0,
                    c->n_head_kv > 1 ? c->head_stride : 0, PageDiv(c->page_size)};
  return MINFER_OK;
}

}  // namespace

extern "C" {

int minfer_rope_prepare(const minfer_rope_spec* spec, minfer_rope_table* out) {
  if (!spec || !out) return MINFER_ERR_ARG;
  const int rot = spec->rot_dim;
  if ((spec->head_dim != 64 && spec->head_dim != 128) || rot < 2 || rot > spec->head_dim || rot % 2)
    return MINFER_ERR_SHAPE;
  const double s = spec->factor;
  const double fast = spec->beta_fast == 0 ? 32 : spec->beta_fast, slow = spec->beta_slow == 0 ? 1 : spec->beta_slow;
  if ((spec->style != MINFER_ROPE_HALF && spec->style != MINFER_ROPE_INTERLEAVED) ||
      spec->scaling < MINFER_ROPE_NONE || spec->scaling > MINFER_ROPE_YARN || !(spec->theta > 1) ||
      !std::isfinite(spec->theta) || !(s > 0) || !std::isfinite(s) || !std::isfinite(spec->attn_factor) ||
      !(fast > 0) || !(slow > 0) || !std::isfinite(fast) || !std::isfinite(slow))
    return MINFER_ERR_ARG;
  if (spec->scaling == MINFER_ROPE_YARN && spec->n_ctx_orig <= 0) return MINFER_ERR_ARG;

  const double two_pi = 6.283185307179586476925;
  double theta = spec->theta;
  if (spec->scaling == MINFER_ROPE_NTK && rot > 2) theta *= std::pow(s, (double)rot / (rot - 2));
  double low = 0, high = 0;
  if (spec->scaling == MINFER_ROPE_YARN) {
    // the pair that turns `turns` times over the original context
    auto pair_of = [&](double turns) {
      return rot * std::log(spec->n_ctx_orig / (turns * two_pi)) / (2 * std::log(theta));
    };
    low = std::fmax(std::floor(pair_of(fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(slow)), rot - 1.0);
  }
  minfer_rope_table t = {};
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot);
    if (spec->scaling == MINFER_ROPE_LINEAR) f /= s;
    if (spec->scaling == MINFER_ROPE_YARN) {
      const double g = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = f / s * g + f * (1 - g);
    }
    if (!std::isfinite(f)) return MINFER_ERR_ARG;
    const double turns = f / two_pi;  // per position; whole turns drop out
    t.turn[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
  }
  t.mscale = (float)(spec->attn_factor != 0                    ? spec->attn_factor
                        : spec->scaling == MINFER_ROPE_YARN && s > 1 ? 0.1 * std::log(s) + 1
                                                                   : 1.0);
  t.head_dim = spec->head_dim;
  t.rot_dim = rot;
  t.style = spec->style;
  *out = t;
  return MINFER_OK;
}

int minfer_op_page_tables(const int32_t* d_len, const int32_t* d_target, int n_req, int page_size,
                          int n_pages, int32_t* d_table, int max_pages, int32_t* d_free,
                          const int32_t* d_n_free, int32_t* d_n_free_out, int32_t* d_start,
                          int32_t* d_pos, int32_t* d_slot, int max_tokens, int* d_status,
                          void* stream) {
  if (!d_len || !d_target || !d_table || !d_free || !d_n_free || !d_n_free_out || !d_start ||
      (max_tokens > 0 && (!d_pos || !d_slot)) || n_req <= 0 || page_size <= 0 || n_pages <= 0 ||
      max_pages <= 0 || max_tokens < 0)
    return MINFER_ERR_ARG;
  if (n_req > kPageTablesMaxReq || !fits31(n_req, max_pages) || !fits31(max_pages, page_size) ||
      !fits31(n_pages, page_size) || max_tokens >= (1 << 30))
    return MINFER_ERR_TOO_LARGE;
  const PageTablesArgs a{d_len,   d_target, n_req,    page_size,    n_pages, max_pages, max_tokens, d_table,
                         d_free,  d_n_free, d_n_free_out, d_start, d_pos,   d_slot,    d_status, PageDiv(page_size)};
  return from_cuda(page_tables_launch(a, static_cast<cudaStream_t>(stream)));
}

int minfer_op_rope_paged_store(const void* d_qkv, int type, int64_t row_stride,
                               const float* d_bias, const float* d_qnorm, const float* d_knorm,
                               float eps, const minfer_rope_table* rope, const int32_t* d_pos,
                               const int32_t* d_slot, int n_tokens, int n_head,
                               const minfer_paged_cache* cache, void* d_q_out, int64_t q_stride,
                               int* d_status, void* stream) {
  RopePagedArgs a;
  const int rc = check_cache(cache, &a.c);
  if (rc != MINFER_OK) return rc;
  if (!d_qkv || !rope || !d_pos || !d_slot || !d_q_out || n_tokens <= 0 || n_head <= 0 ||
      n_head % cache->n_head_kv != 0 || (d_qnorm == nullptr) != (d_knorm == nullptr) || !(eps >= 0))
    return MINFER_ERR_ARG;
  if (n_head > kMaxHeads) return MINFER_ERR_TOO_LARGE;
  if ((type != MINFER_F32 && type != cache->type) || rope->head_dim != cache->head_dim ||
      rope->rot_dim < 2 || rope->rot_dim > cache->head_dim || rope->rot_dim % 2 ||
      (rope->style != MINFER_ROPE_HALF && rope->style != MINFER_ROPE_INTERLEAVED))
    return MINFER_ERR_SHAPE;
  const int64_t q = (int64_t)n_head * cache->head_dim, kv = (int64_t)cache->n_head_kv * cache->head_dim;
  if (!aligned16(d_qkv) || !aligned16(d_q_out) || !aligned16(d_bias) || !aligned16(d_qnorm) ||
      !aligned16(d_knorm) || !stride_ok(row_stride, n_tokens, type) || !stride_ok(q_stride, n_tokens, cache->type) ||
      (n_tokens > 1 && (row_stride < q + 2 * kv || q_stride < q)))
    return MINFER_ERR_ARG;
  const int sms = current_sms();
  if (sms == 0) return MINFER_ERR_CUDA;
  a.qkv = d_qkv;
  a.row_stride = row_stride;
  a.bias = d_bias;
  a.q_norm = d_qnorm;
  a.k_norm = d_knorm;
  a.eps = eps;
  a.pos = d_pos;
  a.slot = d_slot;
  a.n_tokens = n_tokens;
  a.nh = n_head;
  a.q_out = d_q_out;
  a.q_stride = q_stride;
  a.status = d_status;
  a.rope = *rope;
  return from_cuda(rope_paged_launch(a, type, cache->type, sms, static_cast<cudaStream_t>(stream)));
}

int minfer_op_paged_attention_workspace(int n_req, int n_head, const minfer_paged_cache* cache,
                                        int64_t* bytes) {
  PagedCache c;
  const int rc = check_cache(cache, &c);
  if (rc != MINFER_OK) return rc;
  if (!bytes || n_req <= 0 || n_head <= 0 || n_head % c.nkv != 0) return MINFER_ERR_ARG;
  if (n_head > kMaxHeads) return MINFER_ERR_TOO_LARGE;
  const int sms = current_sms();
  if (sms == 0) return MINFER_ERR_CUDA;
  *bytes = paged_attn_workspace(n_head / c.nkv, c.hd, cache->type, sms);
  return MINFER_OK;
}

int minfer_op_paged_attention(const void* d_q, int64_t q_stride, const minfer_paged_cache* cache,
                              const int32_t* d_table, int64_t table_stride, int max_pages,
                              const int32_t* d_len, int n_req, int n_head, float scale, void* d_o,
                              int64_t o_stride, float* d_lse, void* d_workspace,
                              int64_t workspace_bytes, int* d_status, void* stream) {
  PagedAttnArgs a;
  const int rc = check_cache(cache, &a.c);
  if (rc != MINFER_OK) return rc;
  const int64_t q = (int64_t)n_head * cache->head_dim;
  if (!d_q || !d_table || !d_len || !d_o || !d_workspace || n_req <= 0 || n_head <= 0 ||
      n_head % cache->n_head_kv != 0 || max_pages <= 0 || !(scale >= 0) || !std::isfinite(scale))
    return MINFER_ERR_ARG;
  if (!aligned16(d_q) || !aligned16(d_o) || !aligned16(d_workspace) || !stride_ok(q_stride, n_req, cache->type) ||
      !stride_ok(o_stride, n_req, cache->type) || (n_req > 1 && (q_stride < q || o_stride < q || table_stride < max_pages)))
    return MINFER_ERR_ARG;
  if (!fits31(max_pages, cache->page_size) || n_head > kMaxHeads) return MINFER_ERR_TOO_LARGE;
  const int sms = current_sms();
  if (sms == 0) return MINFER_ERR_CUDA;
  if (workspace_bytes < paged_attn_workspace(n_head / a.c.nkv, a.c.hd, cache->type, sms))
    return MINFER_ERR_TOO_LARGE;
  a.q = d_q;
  a.q_stride = q_stride;
  a.table = d_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.len = d_len;
  a.n_req = n_req;
  a.nh = n_head;
  a.scale = scale == 0.f ? 1.0f / std::sqrt((float)cache->head_dim) : scale;
  a.o = d_o;
  a.o_stride = o_stride;
  a.lse = d_lse;
  a.ws = d_workspace;
  a.status = d_status;
  return from_cuda(paged_attn_launch(a, cache->type, sms, static_cast<cudaStream_t>(stream)));
}

int minfer_op_token_logprobs_workspace(int64_t rows, int64_t vocab, int k, int64_t* bytes) {
  if (!bytes || rows <= 0 || vocab <= 0 || k < 0 || k > kLogprobsMaxTop || k > vocab) return MINFER_ERR_ARG;
  if (rows > INT_MAX || vocab > INT_MAX) return MINFER_ERR_TOO_LARGE;
  const int sms = current_sms();
  if (sms == 0) return MINFER_ERR_CUDA;
  *bytes = logprobs_workspace(rows, vocab, k, sms);
  return MINFER_OK;
}

int minfer_op_token_logprobs(const void* d_logits, int type, int64_t rows, int64_t vocab,
                             int64_t row_stride, const int32_t* d_ids, int k, float* d_logprob,
                             float* d_entropy, int32_t* d_top_ids, float* d_top_logprobs,
                             void* d_workspace, int64_t workspace_bytes, int* d_status,
                             void* stream) {
  if (!d_logits || rows <= 0 || vocab <= 0 || k < 0 || k > kLogprobsMaxTop || k > vocab || !d_workspace ||
      (d_ids && !d_logprob) || (k > 0 && (!d_top_ids || !d_top_logprobs)) || (rows > 1 && row_stride < vocab) ||
      row_stride < 0)
    return MINFER_ERR_ARG;
  if (!type_ok(type)) return MINFER_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(d_logits) % type_size(type) || !aligned16(d_workspace)) return MINFER_ERR_ARG;
  if (rows > INT_MAX || vocab > INT_MAX) return MINFER_ERR_TOO_LARGE;
  const int sms = current_sms();
  if (sms == 0) return MINFER_ERR_CUDA;
  if (workspace_bytes < logprobs_workspace(rows, vocab, k, sms)) return MINFER_ERR_TOO_LARGE;
  const LogprobsArgs a{d_logits,  rows,      vocab,     row_stride,     d_ids,       k,
                       d_logprob, d_entropy, d_top_ids, d_top_logprobs, d_workspace, d_status};
  return from_cuda(logprobs_launch(a, type, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
